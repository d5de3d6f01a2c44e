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
// head of 128: 1095 us against 1183 us with 32)
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

// A unit of work before splitting: tiles a0 .. a0 + tiles - 1 of one side (0:
// queries, 1: context) of a sample, for every context head, against b0 .. b1 - 1
// of the other; every tile of those costs `weight` products. kinds: the items made
// of it (each with the same split).
struct Unit {
  int32_t sample, side, a0, tiles, b0, b1, weight;
  std::vector<int32_t> kinds;
};

template <typename F>
void add_units(std::vector<Unit>& u, const Side& a, const Side& b, int side, int per, int weight,
               std::vector<int32_t> kinds, F&& take) {
  for (size_t s = 0; s + 1 < a.first.size(); ++s) {
    const int n = a.first[s + 1] - a.first[s];
    if (!take(n)) continue;
    for (int t = 0; t < n; t += per)
      u.push_back({int32_t(s), side, a.first[s] + t, std::min(per, n - t), b.first[s], b.first[s + 1], weight, kinds});
  }
}

int64_t parts_of(const Unit& x, int64_t cost) {
  const int64_t n = x.b1 - x.b0;
  return std::max<int64_t>(1, std::min<int64_t>(n, (n * x.weight + cost - 1) / cost));
}

// Largest cost of a part: of some candidates the one whose parts, the longest
// first onto `slots` places, end earliest. An item costs its products plus about
// two tiles' for its start and end, a part of a split one about three more for
// its partial result and the join (measured: parts of a ragged batch cut to
// twice the number cost as much as the better balance gained). Parts have at least
// min_len tiles, and batches with many more items than places are not split.
int64_t part_cost(const std::vector<Unit>& u, int groups, int slots, int min_len) {
  int64_t longest = 1, count = 0;
  int weight = 1;
  for (const Unit& x : u) {
    longest = std::max<int64_t>(longest, int64_t(x.b1 - x.b0) * x.weight);
    count += int64_t(x.kinds.size()) * groups;
    weight = std::max<int>(weight, x.weight);
  }
  if (count > 16 * int64_t(slots)) return longest;
  int64_t best = longest, best_end = INT64_MAX;
  for (int64_t parts = 1; parts <= 64; parts += 1 + parts / 8) {
    const int64_t cost = (longest + parts - 1) / parts;
    if (parts > 1 && cost < int64_t(min_len) * weight) break;
    std::vector<int64_t> costs;
    for (const Unit& x : u) {
      const int64_t k = parts_of(x, cost), n = (x.b1 - x.b0 + k - 1) / k;
      costs.insert(costs.end(), size_t(k) * size_t(groups) * x.kinds.size(), (n + (k > 1 ? 5 : 2)) * x.weight);
    }
    if (parts > 1 && int64_t(costs.size()) > 16 * int64_t(slots)) break;
    std::sort(costs.begin(), costs.end(), std::greater<int64_t>());
    std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> ends;
    int64_t end = 0;
    for (int64_t c : costs) {
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
      best = cost;
    }
  }
  return best;
}

// One launch takes all workgroups of a kernel.
void need_launch(int64_t workgroups) {
  if (workgroups > kMaxWorkgroups)
    throw Error{CGTP_ERR_UNSUPPORTED, "attention: more tiles x context heads than one launch takes"};
}

// Splits long units (of at most `stride` tiles) and lays the items out for the
// device. `slots` is the number of workgroups that the device works on at once.
// Order: workgroups go to the 8 dies in turn, and each die has its own L2, so
// all items that read the same packed tiles (one sample, side and context head)
// are given to one die and follow each other there, those with the longest items
// first, so that the short ones fill the end; a group bigger than a die's share
// goes round several.
void build(WorkList& w, const std::vector<Unit>& u, int stride, int groups, int slots, int min_len) {
  int64_t whole = 0;
  for (const Unit& x : u) whole += int64_t(x.kinds.size()) * groups;
  need_launch(whole);  // (before the lists are laid out)
  const int64_t cost = part_cost(u, groups, slots, min_len);
  struct Group {
    int64_t work = 0, longest = 0;
    std::vector<Item> items;
    std::vector<int64_t> costs;
  };
  std::vector<Group> gs;
  std::vector<Join> joins[2];
  int64_t nslot[2] = {0, 0};
  for (size_t i = 0; i < u.size();) {
    size_t j = i;
    while (j < u.size() && u[j].sample == u[i].sample && u[j].side == u[i].side) ++j;
    for (int hk = 0; hk < groups; ++hk) {
      std::vector<Group> g(u[i].kinds.size());
      for (size_t k = i; k < j; ++k) {
        const Unit& x = u[k];
        const int64_t n = x.b1 - x.b0, parts = parts_of(x, cost);
        int64_t& slot = nslot[x.side];
        for (size_t q = 0; q < g.size(); ++q)
          for (int64_t p = 0; p < parts; ++p) {
            const int32_t b0 = int32_t(x.b0 + n * p / parts), b1 = int32_t(x.b0 + n * (p + 1) / parts);
            g[q].items.push_back(
                {x.a0, x.tiles, b0, b1, hk, parts > 1 ? int32_t(slot + p) : -1, stride, x.kinds[q]});
            g[q].costs.push_back(int64_t(b1 - b0 + 1) * x.weight);
            g[q].work += g[q].costs.back();
            g[q].longest = std::max(g[q].longest, g[q].costs.back());
          }
        if (parts > 1) {
          for (int t = 0; t < x.tiles; ++t)
            joins[x.side].push_back({x.a0 + t, hk, int32_t(slot), int32_t(parts), stride, t, 0, 0});
          slot += parts;
        }
      }
      for (Group& q : g) gs.push_back(std::move(q));
    }
    i = j;
  }

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
        const int64_t c = g.costs[at];
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
  need_launch(int64_t(items.size()));
  w.items = int(items.size());
  w.item_mem.upload(items.data(), items.size() * sizeof(Item));
  for (int k = 0; k < 2; ++k) {
    w.part_tiles[k] = nslot[k] * stride;
    if (w.part_tiles[k] > INT32_MAX / 32) throw Error{CGTP_ERR_UNSUPPORTED, "attention: too many partial tiles"};
    w.joins[k] = int(joins[k].size());
    w.join_mem[k].upload(joins[k].data(), joins[k].size() * sizeof(Join));
  }
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
  char *kforms, *qforms;  // at strides of kbytes and qbytes
  size_t kbytes, qbytes;
  float *bias, *rows, *part_q, *part_k, *part_v;
  size_t bytes;
};
Backward carve_backward(const cgtp_attn_batch_s* b, void* p) {
  Carve c{static_cast<char*>(p)};
  const cgtp_attn_s* a = b->attn;
  const size_t g = size_t(a->kv_heads), nk = size_t(b->ktiles) * g * tile_bytes(a);
  const size_t nq = size_t(b->qtiles) * g * tile_bytes(a);
  Backward x{};
  x.kbytes = nk;  // tiles are multiples of 1 KB
  x.qbytes = nq;
  x.kforms = static_cast<char*>(c.take(kKForms * nk));
  x.qforms = static_cast<char*>(c.take(kQForms * nq));
  x.bias = static_cast<float*>(c.take(size_t(b->ktiles) * 32 * 4));
  x.rows = static_cast<float*>(c.take(size_t(b->qtiles) * g * 64 * 4));
  x.part_q = static_cast<float*>(c.take(size_t(b->bwd.part_tiles[0]) * 32 * size_t(a->DP) * 4));
  x.part_k = static_cast<float*>(c.take(size_t(b->bwd.part_tiles[1]) * 32 * size_t(a->DP) * 4));
  x.part_v = static_cast<float*>(c.take(size_t(b->bwd.part_tiles[1]) * 32 * size_t(a->DP) * 4));
  x.bytes = c.used;
  return x;
}

int64_t fwd_part_tiles(const cgtp_attn_batch_s* b) {
  return std::max(std::max(b->fwd.part_tiles[0], b->few.part_tiles[0]), b->wide.part_tiles[0]);
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
  need_launch((std::max(b->qtiles, b->ktiles) + 7) / 8 * 8 * at->kv_heads);  // of the packing
  b->qtile_mem.upload(qs.tiles.data(), qs.tiles.size() * sizeof(Tile));
  b->ktile_mem.upload(ks.tiles.data(), ks.tiles.size() * sizeof(Tile));
  const int g = at->kv_heads;
  // samples with one query tile take the kernel whose waves share the queries,
  // those with enough rows the one of 64 rows a wave
  const int wide = wide_forward(at->DP, dtype_size(at->dtype)) ? kWideTiles : INT32_MAX;
  // workgroups at once: two a compute unit where registers and shared memory allow
  const int es = int(dtype_size(at->dtype)), two = 2 * kCus, one = kCus;
  const int slots = at->DP * es <= 512 ? two : one;
  const auto forward = [&](WorkList& w, int per, int slots, int min_len, auto&& take) {
    std::vector<Unit> u;
    add_units(u, qs, ks, 0, per, 1, {0}, take);
    build(w, u, per, g, slots, min_len);
  };
  forward(b->fwd, 4, slots, 4, [&](int n) { return n > 1 && n < wide; });
  forward(b->wide, 8, two, 4, [&](int n) { return n >= wide; });
  forward(b->few, 1, slots, 8, [](int n) { return n == 1; });
  std::vector<Unit> u;
  const auto all = [](int) { return true; };
  add_units(u, qs, ks, 0, 4, 3, {kItemQ}, all);
  if (one_pass(at->DP, dtype_size(at->dtype)))
    add_units(u, ks, qs, 1, 4, 4, {kItemV}, all);
  else
    add_units(u, ks, qs, 1, 4, 3, {kItemV, kItemK}, all);
  build(b->bwd, u, 4, g, at->DP * es <= 384 ? two : one, 4);
  return b.release();
}

size_t attn_context_bytes(const cgtp_attn_batch_s* b) { return carve_context(b, nullptr).bytes; }

size_t attn_forward_ws_bytes(const cgtp_attn_batch_s* b, bool packed) {
  const size_t part = size_t(fwd_part_tiles(b)) * 32 * (size_t(b->attn->DP) + 4) * 4;
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
  p.size = a->D;
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
  f.part_ml = static_cast<float4*>(ws);
  f.part = reinterpret_cast<float*>(f.part_ml + size_t(fwd_part_tiles(b)) * 32);
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
    f.joins = w.join_mem[0].as<Join>();
    a->k.fwd(f, w.items, tiles, s);
    CGTP_CHECK_HIP(hipGetLastError());
    if (w.joins[0]) {
      a->k.fwd_join(f, w.joins[0], s);
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
    p.t[0].row_frags = w.kforms + kKRows * w.kbytes;
    p.t[0].col_frags = dq ? w.kforms + kKCols * w.kbytes : nullptr;
    p.bias = w.bias;
    p.t[1].row_frags = w.kforms + kVRows * w.kbytes;
    a->k.pack(p, s);
    CGTP_CHECK_HIP(hipGetLastError());
  }
  if (b->qtiles) {
    const bool keys = dk || dv;
    PackArgs p{};
    p.t[0].src = q.p;
    p.t[0].ld = q.ld;
    p.t[0].vec = vec_rows(a, q.p, q.ld);
    p.t[0].row_frags = w.qforms + kQRows * w.qbytes;
    p.t[0].col_frags = keys ? w.qforms + kQCols * w.qbytes : nullptr;
    p.t[1].src = g.p;
    p.t[1].ld = g.ld;
    p.t[1].vec = vec_rows(a, g.p, g.ld);
    p.t[1].row_frags = w.qforms + kGRows * w.qbytes;
    p.t[1].col_frags = keys ? w.qforms + kGCols * w.qbytes : nullptr;
    p.rows_out = w.rows;
    p.tiles = b->qtile_mem.as<Tile>();
    p.table = a->table.as<int4>();
    p.size = a->D;
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
  x.kforms_ = w.kforms;
  x.qforms_ = w.qforms;
  x.kstride = int64_t(w.kbytes / dtype_size(a->dtype));
  x.qstride = int64_t(w.qbytes / dtype_size(a->dtype));
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
  x.part_q = w.part_q;
  x.part_k = w.part_k;
  x.part_v = w.part_v;
  const WorkList& l = b->bwd;
  if (l.items == 0) return;
  x.items = l.item_mem.as<Item>();
  a->k.bwd(x, l.items, s);
  CGTP_CHECK_HIP(hipGetLastError());
  if (dq && l.joins[0]) {
    const GradJoinArgs j{l.join_mem[0].as<Join>(), x.qtiles, x.table, w.part_q, nullptr, dq, nullptr, x.ldq, a->G,
                         true, x.q_quad};
    a->k.grad_join(j, l.joins[0], 1, s);
    CGTP_CHECK_HIP(hipGetLastError());
  }
  if ((dk || dv) && l.joins[1]) {
    GradJoinArgs j{l.join_mem[1].as<Join>(), x.ktiles, x.table, w.part_k, w.part_v, dk, dv, x.ldk, 1, false,
                   x.k_quad};
    if (!dk) {
      j.part0 = j.part1;
      j.dst0 = j.dst1;
    }
    a->k.grad_join(j, l.joins[1], dk && dv ? 2 : 1, s);
    CGTP_CHECK_HIP(hipGetLastError());
  }
}

}  // namespace cgtp
