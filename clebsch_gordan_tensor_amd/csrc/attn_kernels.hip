// Cross attention: handles, work lists and dispatch (kernels: attn_impl.hpp).
#include <algorithm>
#include <cmath>
#include <functional>
#include <numeric>
#include <queue>

#include "attn.hpp"

namespace cgtp {

namespace attn {

KernelTable kernels_f32_a(int dp);
KernelTable kernels_f32_b(int dp);
KernelTable kernels_bf16_a(int dp);
KernelTable kernels_bf16_b(int dp);
KernelTable kernels_f32(int dp) { return dp <= 128 ? kernels_f32_a(dp) : kernels_f32_b(dp); }
KernelTable kernels_bf16(int dp) { return dp <= 128 ? kernels_bf16_a(dp) : kernels_bf16_b(dp); }

namespace {

constexpr int kXcds = 8;
constexpr int kCus = 256;
// query tiles of a sample from which the forward takes 64 rows a wave (long contexts,
// head of 128: 1105 us against 1185 us with 32)
constexpr int kWideTiles = 8;

// One side of a batch cut into 32-row tiles, per sample.
struct Side {
  std::vector<Tile> tiles;
  std::vector<int32_t> first;  // first tile of each sample, [S + 1]
};

Side cut(const std::vector<int64_t>& ptr, int64_t G) {
  Side s;
  if (ptr.back() * G > INT32_MAX - 64) throw Error{CGTP_ERR_UNSUPPORTED, "attention: rows x heads beyond 2^31"};
  for (size_t i = 0; i + 1 < ptr.size(); ++i) {
    s.first.push_back(int32_t(s.tiles.size()));
    const int64_t a = ptr[i] * G, b = ptr[i + 1] * G;
    for (int64_t r = a; r < b; r += 32) s.tiles.push_back({int32_t(r), int32_t(std::min<int64_t>(32, b - r))});
  }
  s.first.push_back(int32_t(s.tiles.size()));
  return s;
}

// A unit of work before splitting: tiles a0 .. a0 + tiles - 1 of one side of
// sample s, for every context head, against b0 .. b1 - 1 of the other.
struct Unit {
  int32_t sample, a0, tiles, b0, b1;
};

template <typename F>
std::vector<Unit> units(const Side& a, const Side& b, int per, F&& take) {
  std::vector<Unit> u;
  for (size_t s = 0; s + 1 < a.first.size(); ++s) {
    const int n = a.first[s + 1] - a.first[s];
    if (!take(n)) continue;
    for (int t = 0; t < n; t += per)
      u.push_back({int32_t(s), a.first[s] + t, std::min(per, n - t), b.first[s], b.first[s + 1]});
  }
  return u;
}

// Longest part of a unit, in tiles: of some candidates the one whose parts, the
// longest first onto `slots` places, end earliest. An item costs its tiles plus
// about two for its start and end, a part of a split one about three more for
// its partial result and the join (measured: parts of a ragged batch cut to
// twice the number cost as much as the better balance gained). Parts have at least
// min_len tiles, and batches with many more items than places are not split.
int64_t part_length(const std::vector<Unit>& u, int groups, int slots, int min_len) {
  int64_t longest = 1;
  for (const Unit& x : u) longest = std::max<int64_t>(longest, x.b1 - x.b0);
  if (int64_t(u.size()) * groups > 16 * int64_t(slots)) return longest;
  int64_t best = longest, best_end = INT64_MAX;
  for (int64_t parts = 1; parts <= 64; parts += 1 + parts / 8) {
    const int64_t len = (longest + parts - 1) / parts;
    if (parts > 1 && len < min_len) break;
    std::vector<int64_t> cost;
    for (const Unit& x : u) {
      const int64_t n = x.b1 - x.b0, k = std::max<int64_t>(1, (n + len - 1) / len);
      for (int64_t i = 0; i < k * groups; ++i) cost.push_back((n + k - 1) / k + (k > 1 ? 5 : 2));
    }
    if (parts > 1 && int64_t(cost.size()) > 16 * int64_t(slots)) break;
    std::sort(cost.begin(), cost.end(), std::greater<int64_t>());
    std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> ends;
    int64_t end = 0;
    for (int64_t c : cost) {
      int64_t t = c;
      if (int64_t(ends.size()) >= slots) {
        t += ends.top();
        ends.pop();
      }
      ends.push(t);
      end = std::max(end, t);
    }
    if (end < best_end) {
      best_end = end;
      best = len;
    }
  }
  return best;
}

// Splits long units (of at most `stride` tiles) and lays the items out for the
// device.
//
// `slots` is the number of workgroups that the device works on at once.
// Order: workgroups go to the 8 dies in turn, and each die has its own L2, so
// all items that read the same packed tiles (one sample and context head) are
// given to one die and follow each other there, those with the longest items
// first, so that the short ones fill the end; a group bigger than a die's share
// goes round several.
void build(WorkList& w, const std::vector<Unit>& u, int stride, int groups, int slots, int min_len) {
  const int64_t len = part_length(u, groups, slots, min_len);
  struct Group {
    int64_t work = 0, longest = 0;
    std::vector<Item> items;
  };
  std::vector<Group> gs;
  std::vector<Join> joins;
  int64_t nslot = 0;
  for (size_t i = 0; i < u.size();) {
    size_t j = i;
    while (j < u.size() && u[j].sample == u[i].sample) ++j;
    for (int hk = 0; hk < groups; ++hk) {
      Group g;
      for (size_t k = i; k < j; ++k) {
        const Unit& x = u[k];
        const int64_t n = x.b1 - x.b0, parts = std::max<int64_t>(1, (n + len - 1) / len);
        for (int64_t p = 0; p < parts; ++p) {
          const int32_t b0 = int32_t(x.b0 + n * p / parts), b1 = int32_t(x.b0 + n * (p + 1) / parts);
          g.items.push_back({x.a0, x.tiles, b0, b1, hk, parts > 1 ? int32_t(nslot + p) : -1, stride, 0});
          g.work += b1 - b0 + 1;
          g.longest = std::max<int64_t>(g.longest, b1 - b0);
        }
        if (parts > 1) {
          for (int t = 0; t < x.tiles; ++t)
            joins.push_back({x.a0 + t, hk, int32_t(nslot), int32_t(parts), stride, t, 0, 0});
          nslot += parts;
        }
      }
      gs.push_back(std::move(g));
    }
    i = j;
  }
  w.part_tiles = nslot * stride;
  if (w.part_tiles > INT32_MAX / 32) throw Error{CGTP_ERR_UNSUPPORTED, "attention: too many partial tiles"};

  int64_t total = 0;
  for (const Group& g : gs) total += g.work;
  const int64_t share = std::max<int64_t>(1, total / kXcds);
  std::vector<std::vector<Item>> queue(kXcds);
  std::vector<int64_t> load(kXcds, 0);
  std::vector<size_t> order(gs.size());
  std::iota(order.begin(), order.end(), size_t(0));
  std::stable_sort(order.begin(), order.end(), [&](size_t a, size_t b) { return gs[a].longest > gs[b].longest; });
  for (size_t gi : order) {
    const Group& g = gs[gi];
    size_t at = 0;
    while (at < g.items.size()) {
      const int x = int(std::min_element(load.begin(), load.end()) - load.begin());
      int64_t room = std::max<int64_t>(1, share - load[x]);
      while (at < g.items.size() && room > 0) {
        const int64_t c = g.items[at].b1 - g.items[at].b0 + 1;
        queue[size_t(x)].push_back(g.items[at++]);
        load[size_t(x)] += c;
        room -= c;
      }
    }
  }
  size_t longest = 0;
  for (const auto& q : queue) longest = std::max(longest, q.size());
  std::vector<Item> items;
  for (size_t k = 0; k < longest; ++k)
    for (int x = 0; x < kXcds; ++x)
      items.push_back(k < queue[size_t(x)].size() ? queue[size_t(x)][k] : Item{0, 0, 0, 0, 0, -1, stride, 0});
  // trailing empty places of the last turn
  while (!items.empty() && items.back().tiles == 0) items.pop_back();
  if (items.size() > size_t(INT32_MAX)) throw Error{CGTP_ERR_UNSUPPORTED, "attention: too many work items"};
  w.items = int(items.size());
  w.joins = int(joins.size());
  w.item_mem.upload(items.data(), items.size() * sizeof(Item));
  w.join_mem.upload(joins.data(), joins.size() * sizeof(Join));
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Carve {
  char* p;
  size_t used = 0;
  void* take(size_t n) {
    void* r = p ? p + used : nullptr;
    used += up16(n);
    return r;
  }
};

size_t tile_bytes(const cgtp_attn_s* a) { return size_t(a->DP) * 32 * dtype_size(a->dtype); }

// Packed context: key row fragments, value column fragments, key biases.
struct Context {
  void *kf, *vf;
  float *bias, *norms;
  int32_t* flags;
  size_t bytes;
};
Context carve_context(const cgtp_attn_batch_s* b, void* p) {
  Carve c{static_cast<char*>(p)};
  const size_t n = size_t(b->ktiles) * size_t(b->attn->kv_heads) * tile_bytes(b->attn);
  Context x{};
  x.kf = c.take(n);
  x.vf = c.take(n);
  x.bias = static_cast<float*>(c.take(size_t(b->ktiles) * 32 * 4));
  x.norms = static_cast<float*>(c.take(size_t(b->ktiles) * size_t(b->attn->kv_heads) * 4));
  x.flags = static_cast<int32_t*>(c.take(size_t(b->ktiles) * 4));
  x.bytes = c.used;
  return x;
}

struct Backward {
  void *kr, *kc, *vr, *qr, *qc, *gr, *gc;
  float *bias, *rows, *part_q, *part_k, *part_v;
  size_t bytes;
};
Backward carve_backward(const cgtp_attn_batch_s* b, void* p) {
  Carve c{static_cast<char*>(p)};
  const cgtp_attn_s* a = b->attn;
  const size_t g = size_t(a->kv_heads), nk = size_t(b->ktiles) * g * tile_bytes(a);
  const size_t nq = size_t(b->qtiles) * g * tile_bytes(a);
  Backward x{};
  x.kr = c.take(nk);
  x.kc = c.take(nk);
  x.vr = c.take(nk);
  x.qr = c.take(nq);
  x.qc = c.take(nq);
  x.gr = c.take(nq);
  x.gc = c.take(nq);
  x.bias = static_cast<float*>(c.take(size_t(b->ktiles) * 32 * 4));
  x.rows = static_cast<float*>(c.take(size_t(b->qtiles) * g * 64 * 4));
  x.part_q = static_cast<float*>(c.take(size_t(b->dq.part_tiles) * 32 * size_t(a->DP) * 4));
  x.part_k = static_cast<float*>(c.take(size_t(b->dkv.part_tiles) * 32 * size_t(a->DP) * 4));
  x.part_v = static_cast<float*>(c.take(size_t(b->dkv.part_tiles) * 32 * size_t(a->DP) * 4));
  x.bytes = c.used;
  return x;
}

int64_t fwd_part_tiles(const cgtp_attn_batch_s* b) {
  return std::max(std::max(b->fwd.part_tiles, b->few.part_tiles), b->wide.part_tiles);
}

}  // namespace
}  // namespace attn

using namespace attn;

cgtp_attn_s* build_attn(const char* irreps, int64_t heads, int64_t kv_heads, cgtp_dtype dtype) {
  if (dtype == CGTP_F64) throw Error{CGTP_ERR_UNSUPPORTED, "attention: fp64 is not supported (fp32, bf16)"};
  if (dtype != CGTP_F32 && dtype != CGTP_BF16) throw Error{CGTP_ERR_INVALID_ARG, "bad dtype"};
  if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0)
    throw Error{CGTP_ERR_INVALID_ARG, "attention: kv_heads must divide heads (both at least 1)"};
  auto a = std::make_unique<cgtp_attn_s>();
  a->qrow = row_layout(irreps);
  for (const Irrep& i : a->qrow.irreps)
    if (heads > i.mul || i.mul % heads != 0)
      throw Error{CGTP_ERR_UNSUPPORTED, "attention: heads must divide every multiplicity"};
  a->heads = int(heads);
  a->kv_heads = int(kv_heads);
  a->G = int(heads / kv_heads);
  a->dtype = dtype;
  const int64_t D = a->qrow.dim / heads;
  if (D > 256) throw Error{CGTP_ERR_UNSUPPORTED, "attention: more than 256 elements a head"};
  a->D = int(D);
  a->DP = (a->D + 31) / 32 * 32;
  std::string kv;
  for (const Irrep& i : a->qrow.irreps)
    kv += (kv.empty() ? "" : "+") + std::to_string(i.mul / a->G) + "x" + std::to_string(i.l) + (i.p > 0 ? "e" : "o");
  a->krow = row_layout(kv.c_str());
  const int ve = 16 / int(dtype_size(dtype));
  a->vec16 = a->quad = true;
  std::vector<int4> table;
  for (size_t i = 0; i < a->qrow.blocks.size(); ++i) {
    const RowBlock &q = a->qrow.blocks[i], &k = a->krow.blocks[i];
    const int cw = q.mul / a->heads;
    a->vec16 = a->vec16 && cw % ve == 0;
    a->quad = a->quad && cw % 4 == 0;
    for (int m = 0; m < q.nc; ++m)
      for (int c = 0; c < cw; ++c) table.push_back({q.off + m * q.mul + c, k.off + m * k.mul + c, cw, 1});
  }
  table.resize(size_t(a->DP), int4{0, 0, 0, 0});
  a->k = dtype == CGTP_BF16 ? kernels_bf16(a->DP) : kernels_f32(a->DP);
  a->device = current_device();
  a->table.upload(table.data(), table.size() * sizeof(int4));
  return a.release();
}

cgtp_attn_batch_s* build_attn_batch(cgtp_attn_s* at, const cgtp_samples_s* q, const cgtp_samples_s* k) {
  if (q->S != k->S) throw Error{CGTP_ERR_INVALID_ARG, "attention: the two sides have different numbers of samples"};
  auto b = std::make_unique<cgtp_attn_batch_s>();
  b->attn = at;
  b->nq = q->rows;
  b->nk = k->rows;
  b->device = current_device();
  const Side qs = cut(q->ptr, at->G), ks = cut(k->ptr, 1);
  b->qtiles = int64_t(qs.tiles.size());
  b->ktiles = int64_t(ks.tiles.size());
  b->qtile_mem.upload(qs.tiles.data(), qs.tiles.size() * sizeof(Tile));
  b->ktile_mem.upload(ks.tiles.data(), ks.tiles.size() * sizeof(Tile));
  const int g = at->kv_heads;
  // samples with one query tile take the kernel whose waves share the queries,
  // those with enough rows the one of 64 rows a wave
  const int wide = wide_forward(at->DP, dtype_size(at->dtype)) ? kWideTiles : INT32_MAX;
  // workgroups at once: two a compute unit where registers and shared memory allow
  const int es = int(dtype_size(at->dtype)), two = 2 * kCus, one = kCus;
  const int slots = at->DP * es <= 512 ? two : one;
  build(b->fwd, units(qs, ks, 4, [&](int n) { return n > 1 && n < wide; }), 4, g, slots, 4);
  build(b->wide, units(qs, ks, 8, [&](int n) { return n >= wide; }), 8, g, two, 4);
  build(b->few, units(qs, ks, 1, [](int n) { return n == 1; }), 1, g, slots, 8);
  const int bslots = at->DP * es <= 384 ? two : one;
  build(b->dq, units(qs, ks, 4, [](int) { return true; }), 4, g, bslots, 4);
  build(b->dkv, units(ks, qs, 4, [](int) { return true; }), 4, g, bslots, 4);
  return b.release();
}

size_t attn_context_bytes(const cgtp_attn_batch_s* b) { return carve_context(b, nullptr).bytes; }

size_t attn_forward_ws_bytes(const cgtp_attn_batch_s* b, bool packed) {
  const size_t part = size_t(fwd_part_tiles(b)) * 32 * (size_t(b->attn->DP) + 2) * 4;
  return up16(part) + (packed ? 0 : attn_context_bytes(b));
}

size_t attn_backward_ws_bytes(const cgtp_attn_batch_s* b) { return carve_backward(b, nullptr).bytes; }

namespace {

bool vec_rows(const cgtp_attn_s* a, const void* p, int64_t ld) {
  return a->vec16 && aligned(p, 16) && (ld * int64_t(dtype_size(a->dtype))) % 16 == 0;
}
// four-element stores
bool quad_rows(const cgtp_attn_s* a, const void* p) {
  return a->quad && aligned(p, 4 * dtype_size(a->dtype));
}

PackArgs context_pack(const cgtp_attn_batch_s* b, RowsIn k, RowsIn v, const uint8_t* mask) {
  const cgtp_attn_s* a = b->attn;
  PackArgs p{};
  p.t[0].src = k.p;
  p.t[0].ld = k.ld;
  p.t[0].vec = vec_rows(a, k.p, k.ld);
  p.t[1].src = v.p;
  p.t[1].ld = v.ld;
  p.t[1].vec = vec_rows(a, v.p, v.ld);
  p.tiles = b->ktile_mem.as<Tile>();
  p.ntiles = int(b->ktiles);
  p.table = a->table.as<int4>();
  p.mask = mask;
  p.heads = a->heads;
  p.groups = a->kv_heads;
  return p;
}

}  // namespace

void attn_pack_launch(const cgtp_attn_batch_s* b, RowsIn k, RowsIn v, const uint8_t* mask, void* context,
                      hipStream_t s) {
  if (b->ktiles == 0) return;
  const Context c = carve_context(b, context);
  PackArgs p = context_pack(b, k, v, mask);
  p.t[0].row_frags = c.kf;
  p.bias = c.bias;
  p.flags = c.flags;
  p.norms = c.norms;
  p.t[1].col_frags = c.vf;
  b->attn->k.pack(p, s);
  CGTP_CHECK_HIP(hipGetLastError());
}

void attn_forward_launch(const cgtp_attn_batch_s* b, RowsIn q, const void* context, double scale, void* out,
                         float* lse, void* ws, hipStream_t s) {
  const cgtp_attn_s* a = b->attn;
  const Context c = carve_context(b, const_cast<void*>(context));
  FwdArgs f{};
  f.qtiles = b->qtile_mem.as<Tile>();
  f.table = a->table.as<int4>();
  f.q = q.p;
  f.ldq = q.ld;
  f.q_vec = vec_rows(a, q.p, q.ld);
  f.kf = c.kf;
  f.vf = c.vf;
  f.bias = c.bias;
  f.flags = c.flags;
  f.norms = c.norms;
  f.out = out;
  f.ldo = a->qrow.dim;
  f.out_quad = quad_rows(a, out);
  f.lse = lse;
  f.part_ml = static_cast<float*>(ws);
  f.part = f.part_ml + size_t(fwd_part_tiles(b)) * 64;
  // a zero scale stays a small positive one: every score is then 0 all the same
  f.scale2 = std::max(float(std::fabs(scale) * 1.4426950408889634), 1e-37f);
  f.q_sign = scale < 0.0 ? (a->dtype == CGTP_BF16 ? 0x80008000u : 0x80000000u) : 0u;
  f.G = a->G;
  f.heads = a->heads;
  f.groups = a->kv_heads;
  // the lists share the partial buffers: each is joined before the next starts
  for (const int tiles : {8, 4, 1}) {
    const WorkList& w = tiles == 8 ? b->wide : tiles == 4 ? b->fwd : b->few;
    if (w.items == 0) continue;
    f.items = w.item_mem.as<Item>();
    f.joins = w.join_mem.as<Join>();
    a->k.fwd(f, w.items, tiles, s);
    CGTP_CHECK_HIP(hipGetLastError());
    if (w.joins) {
      a->k.fwd_join(f, w.joins, s);
      CGTP_CHECK_HIP(hipGetLastError());
    }
  }
}

void attn_backward_launch(const cgtp_attn_batch_s* b, RowsIn q, RowsIn k, RowsIn v, const uint8_t* mask, double scale,
                          const void* out, const float* lse, RowsIn g, void* dq, void* dk, void* dv, void* ws,
                          hipStream_t s) {
  const cgtp_attn_s* a = b->attn;
  const Backward w = carve_backward(b, ws);
  if (b->ktiles) {
    PackArgs p = context_pack(b, k, v, mask);
    p.t[0].row_frags = w.kr;
    p.t[0].col_frags = dq ? w.kc : nullptr;
    p.bias = w.bias;
    p.t[1].row_frags = w.vr;
    a->k.pack(p, s);
    CGTP_CHECK_HIP(hipGetLastError());
  }
  if (b->qtiles) {
    const bool keys = dk || dv;
    PackArgs p{};
    p.t[0].src = q.p;
    p.t[0].ld = q.ld;
    p.t[0].vec = vec_rows(a, q.p, q.ld);
    p.t[0].row_frags = w.qr;
    p.t[0].col_frags = keys ? w.qc : nullptr;
    p.t[1].src = g.p;
    p.t[1].ld = g.ld;
    p.t[1].vec = vec_rows(a, g.p, g.ld);
    p.t[1].row_frags = w.gr;
    p.t[1].col_frags = keys ? w.gc : nullptr;
    p.rows_out = w.rows;
    p.tiles = b->qtile_mem.as<Tile>();
    p.table = a->table.as<int4>();
    p.out = out;
    p.ldo = a->qrow.dim;
    p.out_vec = vec_rows(a, out, a->qrow.dim);
    p.lse = lse;
    p.G = a->G;
    p.heads = a->heads;
    p.groups = a->kv_heads;
    p.ntiles = int(b->qtiles);
    a->k.pack(p, s);
    CGTP_CHECK_HIP(hipGetLastError());
  }
  BwdArgs x{};
  x.qtiles = b->qtile_mem.as<Tile>();
  x.ktiles = b->ktile_mem.as<Tile>();
  x.table = a->table.as<int4>();
  x.kr = w.kr;
  x.kc = w.kc;
  x.vr = w.vr;
  x.qr = w.qr;
  x.qc = w.qc;
  x.gr = w.gr;
  x.gc = w.gc;
  x.bias = w.bias;
  x.rows = w.rows;
  x.dq = dq;
  x.dk = dk;
  x.dv = dv;
  x.ldq = a->qrow.dim;
  x.ldk = a->krow.dim;
  x.q_quad = dq && quad_rows(a, dq);
  x.k_quad = (!dk || quad_rows(a, dk)) && (!dv || quad_rows(a, dv));
  x.scale = float(scale);
  x.scale2 = float(scale * 1.4426950408889634);
  x.G = a->G;
  x.heads = a->heads;
  x.groups = a->kv_heads;
  if (dq && b->dq.items) {
    x.items = b->dq.item_mem.as<Item>();
    x.part = w.part_q;
    a->k.dq(x, b->dq.items, s);
    CGTP_CHECK_HIP(hipGetLastError());
    if (b->dq.joins) {
      const GradJoinArgs j{b->dq.join_mem.as<Join>(), x.qtiles, x.table, w.part_q, nullptr, dq, nullptr, x.ldq, a->G,
                           true, x.q_quad};
      a->k.grad_join(j, b->dq.joins, 1, s);
      CGTP_CHECK_HIP(hipGetLastError());
    }
  }
  if ((dk || dv) && b->dkv.items) {
    x.items = b->dkv.item_mem.as<Item>();
    x.part = w.part_k;
    x.part_v = w.part_v;
    a->k.dkv(x, b->dkv.items, s);
    CGTP_CHECK_HIP(hipGetLastError());
    if (b->dkv.joins) {
      GradJoinArgs j{b->dkv.join_mem.as<Join>(), x.ktiles, x.table, w.part_k, w.part_v, dk, dv, x.ldk, 1, false,
                     x.k_quad};
      if (!dk) {
        j.part0 = j.part1;
        j.dst0 = j.dst1;
      }
      a->k.grad_join(j, b->dkv.joins, dk && dv ? 2 : 1, s);
      CGTP_CHECK_HIP(hipGetLastError());
    }
  }
}

}  // namespace cgtp
