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
SeqTable seq_kernels_f32_a(int dp);
SeqTable seq_kernels_f32_b(int dp);
SeqTable seq_kernels_bf16_a(int dp);
SeqTable seq_kernels_bf16_b(int dp);
SeqTable seq_kernels_f32(int dp) { return dp <= 128 ? seq_kernels_f32_a(dp) : seq_kernels_f32_b(dp); }
SeqTable seq_kernels_bf16(int dp) { return dp <= 128 ? seq_kernels_bf16_a(dp) : seq_kernels_bf16_b(dp); }

namespace {

constexpr int kXcds = 8;
constexpr int kCus = 256;
// query tiles of a sample from which the forward takes 64 rows a wave (long contexts,
// head of 128: 1095 us against 1183 us with 32)
constexpr int kWideTiles = 8;

// Key tiles up to which a query tile's rows see few keys (delta_kernel: a wave each).
constexpr int kFewKeyTiles = 2;

// One side of a batch cut into 32-row tiles, per sample, after those of `shared` rows
// that come before the samples'.
struct Side {
  std::vector<Tile> tiles;
  std::vector<int32_t> first;  // first tile of each sample, [S + 1]
};

// One launch takes all workgroups of a kernel.
void need_launch(int64_t workgroups) {
  if (workgroups > kMaxWorkgroups)
    throw Error{CGTP_ERR_UNSUPPORTED, "attention: more tiles x context heads than one launch takes"};
}
// That of the packing: checked before the tiles are laid out.
void need_packing(int64_t tiles, int64_t kv_heads) { need_launch((tiles + 7) / 8 * 8 * kv_heads); }

// `kv_heads` > 0: the side is packed by one launch.
Side cut(const std::vector<int64_t>& ptr, int64_t G, int64_t shared = 0, int64_t kv_heads = 0) {
  Side s;
  if (ptr.back() * G + shared > INT32_MAX - 64)
    throw Error{CGTP_ERR_UNSUPPORTED, "attention: rows x heads beyond 2^31"};
  int64_t tiles = (shared + 31) / 32;
  for (size_t i = 0; i + 1 < ptr.size(); ++i) tiles += ((ptr[i + 1] - ptr[i]) * G + 31) / 32;
  need_packing(tiles, kv_heads);
  s.tiles.reserve(size_t(tiles));
  for (int64_t r = 0; r < shared; r += 32) s.tiles.push_back({int32_t(r), int32_t(std::min<int64_t>(32, shared - r))});
  for (size_t i = 0; i + 1 < ptr.size(); ++i) {
    s.first.push_back(int32_t(s.tiles.size()));
    const int64_t a = shared + ptr[i] * G, b = shared + ptr[i + 1] * G;
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

// How the queries of a sequence batch see the context: key tiles of shared rows, and
// whether a query's own keys end with its place (Reach).
struct Sight {
  const std::vector<int64_t>&qptr, &kptr;
  const Side &q, &k;
  int64_t G, shared_tiles;
  bool causal;
  // own keys of sample s, counted from its first, that query token i of the sample sees
  int64_t seen(size_t s, int64_t i) const {
    const int64_t nq = qptr[s + 1] - qptr[s], nk = kptr[s + 1] - kptr[s];
    return causal ? std::max<int64_t>(0, std::min(nk, i + nk - nq + 1)) : nk;
  }
  int32_t skip(size_t s) const { return shared_tiles ? int32_t(k.first[s] - shared_tiles) : 0; }
  Reach reach(size_t s) const {
    const int64_t nq = qptr[s + 1] - qptr[s], nk = kptr[s + 1] - kptr[s];
    return {skip(s), int32_t(32 * int64_t(k.first[s]) + nk - nq + 1 - qptr[s])};
  }
};

// Query tiles against the keys that some query of a unit sees: shared and own ones
// (`own_only`: those alone). Longest units first: in a causal sample the last.
template <typename F>
void add_query_units(std::vector<Unit>& u, const Sight& v, int per, int weight, int32_t kind, bool own_only, F&& take) {
  for (size_t s = 0; s + 1 < v.q.first.size(); ++s) {
    const int n = v.q.first[s + 1] - v.q.first[s];
    if (n == 0 || !take(n)) continue;
    for (int t = (n - 1) / per * per; t >= 0; t -= per) {
      const int tiles = std::min(per, n - t);
      const Tile& last = v.q.tiles[size_t(v.q.first[s] + t + tiles - 1)];
      const int64_t token = (last.row0 + last.n - 1) / v.G - v.qptr[s];
      const int32_t own0 = v.k.first[s] - v.skip(s);  // in the numbering of work lists
      u.push_back({int32_t(s), 0, v.q.first[s] + t, tiles, v.shared_tiles && !own_only ? 0 : own0,
                   own0 + int32_t((v.seen(s, token) + 31) / 32), weight, {kind}});
    }
  }
}

// Key tiles against the query tiles that see some of their keys: those of shared rows
// (as one more sample) against all, every sample's own against those from the first
// query on that sees the first key.
void add_key_units(std::vector<Unit>& u, const Sight& v, int per, int weight, const std::vector<int32_t>& kinds) {
  const int S = int(v.q.first.size()) - 1;
  for (int t = 0; t < v.shared_tiles; t += per)
    u.push_back({S, 1, t, int(std::min<int64_t>(per, v.shared_tiles - t)), 0, v.q.first[size_t(S)], weight, kinds});
  for (size_t s = 0; s < size_t(S); ++s) {
    const int n = v.k.first[s + 1] - v.k.first[s];
    const int64_t nq = v.qptr[s + 1] - v.qptr[s], nk = v.kptr[s + 1] - v.kptr[s];
    for (int t = 0; t < n; t += per) {
      const int64_t i = v.causal ? std::max<int64_t>(0, 32 * int64_t(t) - (nk - nq)) : 0;
      const int32_t end = v.q.first[s + 1];
      const int32_t b0 = i >= nq ? end : v.q.first[s] + int32_t(i * v.G / 32);
      u.push_back({int32_t(s), 1, v.k.first[s] + t, std::min(per, n - t), b0, end, weight, kinds});
    }
  }
}

int64_t parts_of(const Unit& x, int64_t cost) {
  const int64_t n = x.b1 - x.b0;
  return std::max<int64_t>(1, std::min<int64_t>(n, (n * x.weight + cost - 1) / cost));
}

// Largest cost of a part: of some candidates the one whose parts, the longest
// first onto `slots` places, end earliest. An item costs its products plus about
// two tiles' for its start and end, a part of a split one `part_extra` for these, its
// partial result and the join (5 of batches whose samples' queries all see the same
// keys; measured: parts of a ragged batch cut to twice the number cost as much as the better balance gained). Parts have at least
// min_len tiles, and batches with many more items than places are not split.
int64_t part_cost(const std::vector<Unit>& u, int groups, int slots, int min_len, int part_extra, bool sequence) {
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
      costs.insert(costs.end(), size_t(k) * size_t(groups) * x.kinds.size(), (n + (k > 1 ? part_extra : 2)) * x.weight);
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
    // (sequences: near enough to an even share of everything; long prompts are planned in 0.75 ms so)
    if (sequence && best_end * slots * 32 <= std::accumulate(costs.begin(), costs.end(), int64_t(0)) * 33) break;
  }
  return best;
}

// Splits long units (of at most `stride` tiles) and lays the items out for the
// device. `slots` is the number of workgroups that the device works on at once.
// Order: workgroups go to the 8 dies in turn, and each die has its own L2, so
// all items that read the same packed tiles (one sample, side and context head)
// are given to one die and follow each other there, those with the longest items
// first, so that the short ones fill the end; a group bigger than a die's share
// goes round several.
// Returns the largest number of parts of a unit.
struct How {
  bool all_parts = false;  // every result is a part, also that of an unsplit unit
  bool uneven = false;     // the items of a group differ in length (causal queries)
  bool spread = false;     // and go to the dies one by one, not in runs of a group
  int part_extra = 5;      // of part_cost
  int64_t cost = 0;        // largest cost of a part, where it is known
  bool sequence = false;   // of a sequence batch
};
int64_t build(WorkList& w, const std::vector<Unit>& u, int stride, int groups, int slots, int min_len,
              const How& how = {}) {
  int64_t whole = 0;
  for (const Unit& x : u) whole += int64_t(x.kinds.size()) * groups;
  need_launch(whole);  // (before the lists are laid out)
  const int64_t cost = how.cost ? how.cost : part_cost(u, groups, slots, min_len, how.part_extra, how.sequence);
  struct Group {
    int64_t work = 0, longest = 0;
    std::vector<Item> items;
    std::vector<int64_t> costs;
  };
  std::vector<Group> gs;
  std::vector<Join> joins[2];
  int64_t nslot[2] = {0, 0}, most = 1;
  for (size_t i = 0; i < u.size();) {
    size_t j = i;
    while (j < u.size() && u[j].sample == u[i].sample && u[j].side == u[i].side) ++j;
    for (int hk = 0; hk < groups; ++hk) {
      std::vector<Group> g(u[i].kinds.size());
      for (size_t k = i; k < j; ++k) {
        const Unit& x = u[k];
        const int64_t n = x.b1 - x.b0, parts = parts_of(x, cost);
        const bool split = how.all_parts || parts > 1;
        most = std::max(most, parts);
        int64_t& slot = nslot[x.side];
        for (size_t q = 0; q < g.size(); ++q)
          for (int64_t p = 0; p < parts; ++p) {
            const int32_t b0 = int32_t(x.b0 + n * p / parts), b1 = int32_t(x.b0 + n * (p + 1) / parts);
            g[q].items.push_back(
                {x.a0, x.tiles, b0, b1, hk, split ? int32_t(slot + p) : -1, stride, x.kinds[q]});
            g[q].costs.push_back(int64_t(b1 - b0 + 1) * x.weight);
            g[q].work += g[q].costs.back();
            g[q].longest = std::max(g[q].longest, g[q].costs.back());
          }
        if (split) {
          for (int t = 0; t < x.tiles; ++t)
            joins[x.side].push_back({x.a0 + t, hk, int32_t(slot), int32_t(parts), stride, t, 0, 0});
          slot += parts;
        }
      }
      for (Group& q : g) gs.push_back(std::move(q));
    }
    i = j;
  }

  // long and short items in turn, so that every run of them has alike shares of both, and
  // then every die's longest first (long causal prompts 782 us without, 744 us with both)
  if (how.uneven && !how.spread)
    for (Group& g : gs) {
      std::vector<size_t> by(g.items.size());
      std::iota(by.begin(), by.end(), size_t(0));
      std::stable_sort(by.begin(), by.end(), [&](size_t a, size_t b) { return g.costs[a] > g.costs[b]; });
      Group mixed = g;
      for (size_t k = 0; k < by.size(); ++k) {
        const size_t from = k % 2 == 0 ? by[k / 2] : by[by.size() - 1 - k / 2];
        mixed.items[k] = g.items[from];
        mixed.costs[k] = g.costs[from];
      }
      g = std::move(mixed);
    }
  int64_t total = 0;
  for (const Group& g : gs) total += g.work;
  const int64_t share = std::max<int64_t>(1, total / kXcds);
  std::vector<std::vector<Item>> queue(kXcds);
  std::vector<std::vector<int64_t>> queue_costs(kXcds);
  std::vector<int64_t> load(kXcds, 0);
  std::vector<size_t> order(gs.size());
  std::iota(order.begin(), order.end(), size_t(0));
  std::stable_sort(order.begin(), order.end(), [&](size_t a, size_t b) { return gs[a].longest > gs[b].longest; });
  // Gradients: the longest item to the least loaded die (us with and without: one fp32
  // trajectory 510 and 534, a training batch with shared rows 276 and 288; the forward's
  // chunk after earlier rows 157 and 154)
  if (how.spread) {
    std::vector<std::pair<int64_t, const Item*>> all;
    for (size_t gi : order)
      for (size_t k = 0; k < gs[gi].items.size(); ++k) all.push_back({gs[gi].costs[k], &gs[gi].items[k]});
    std::stable_sort(all.begin(), all.end(), [](const auto& a, const auto& b) { return a.first > b.first; });
    for (const auto& x : all) {
      const size_t d = size_t(std::min_element(load.begin(), load.end()) - load.begin());
      queue[d].push_back(*x.second);
      load[d] += x.first;
    }
    order.clear();
  }
  for (size_t gi : order) {
    const Group& g = gs[gi];
    size_t at = 0;
    while (at < g.items.size()) {
      const int x = int(std::min_element(load.begin(), load.end()) - load.begin());
      int64_t room = std::max<int64_t>(1, share - load[x]);
      while (at < g.items.size() && room > 0) {
        const int64_t c = g.costs[at];
        queue[size_t(x)].push_back(g.items[at++]);
        queue_costs[size_t(x)].push_back(c);
        load[size_t(x)] += c;
        room -= c;
      }
    }
  }
  if (how.uneven && !how.spread)
    for (size_t x = 0; x < size_t(kXcds); ++x) {
      std::vector<size_t> by(queue[x].size());
      std::iota(by.begin(), by.end(), size_t(0));
      std::stable_sort(by.begin(), by.end(), [&](size_t a, size_t b) { return queue_costs[x][a] > queue_costs[x][b]; });
      std::vector<Item> sorted;
      for (size_t k : by) sorted.push_back(queue[x][k]);
      queue[x] = std::move(sorted);
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
  if (!items.empty()) w.item_mem.upload(items.data(), items.size() * sizeof(Item));
  for (int k = 0; k < 2; ++k) {
    w.part_tiles[k] = nslot[k] * stride;
    if (w.part_tiles[k] > INT32_MAX / 32) throw Error{CGTP_ERR_UNSUPPORTED, "attention: too many partial tiles"};
    w.joins[k] = int(joins[k].size());
    if (!joins[k].empty()) w.join_mem[k].upload(joins[k].data(), joins[k].size() * sizeof(Join));
  }
  return most;
}

// Workgroups of the forward at once: two a compute unit where registers and shared
// memory allow.
int forward_slots(const cgtp_attn_s* at) { return at->DP * int(dtype_size(at->dtype)) <= 512 ? 2 * kCus : kCus; }

// A part's start, end, partial result and join in tiles of its keys, for sequence
// batches. In bf16 the partial result of 128 or 256 rows (16 KB for every 32 columns of 128
// rows, written and read) costs as much as some twenty tiles' products (us with 5, 12, 24: long
// causal prompts 744, 679, 677; a chunk after earlier rows 202, 202, 154; prompts with a shared
// beginning 335, 335, 318; a chunk of heads of 96 118, 117, 114, of 192 172, 171, 158; prompts of heads of
// 256 341, 246, 246), but for narrow heads, whose exponentials take as long as wide ones' beside
// smaller parts, less (heads of 16, 48 and 64 with 12 and 24: a chunk 58 and 73, 87 and 89, 90 and 91;
// prompts with a shared beginning 141 and 171, 217 and 256, 222 and 255). Products in fp32 take
// eight times as long, and the rows of one tile are few.
int part_extra(const cgtp_attn_s* at, int per) {
  return dtype_size(at->dtype) != 2 || per == 1 ? 5 : at->DP <= 64 ? 12 : 24;
}

// The rows of `tokens` tokens in tiles whatever their sample, against shared_tiles key
// tiles, in items of up to `per` tiles of rows. All units see the same tiles, so they have
// equally many parts: as many as make the turns (about 1 us for 128 elements in bf16, 3.5 us
// in fp32) and the parts' bytes, written and read, the least (64 tokens on 8000 shared rows: 35 of
// a device's 62 parts).
void build_joint(JointPlan& j, const cgtp_attn_s* at, int64_t tokens, int64_t shared_tiles, bool with_step) {
  const Side rows = cut({0, tokens}, at->G);
  const int n = int(rows.tiles.size());
  if (n == 0) return;
  const size_t es = dtype_size(at->dtype);
  j.per = with_step ? 4 : n == 1 ? 1 : n >= kWideTiles && wide_forward(at->DP, es) ? 8 : 4;
  j.units = (n + j.per - 1) / j.per;
  j.tiles.upload(rows.tiles.data(), rows.tiles.size() * sizeof(Tile));
  std::vector<Unit> u;
  for (int t = 0; t < n; t += j.per)
    u.push_back({0, 0, t, std::min(j.per, n - t), 0, int32_t(shared_tiles), 1, {0}});
  const int slots = j.per == 8 ? 2 * kCus : forward_slots(at);
  const double turn = (es == 2 ? 1.0 : 3.5) * at->DP / 128 * (j.per == 8 ? 2 : 1);
  const double part = double(n) * 32 * at->kv_heads * at->DP * 8 / 5e6;  // us
  How how{true, false, false, 0, shared_tiles};
  double best = 1e30;
  for (int64_t p = 1; p <= std::min<int64_t>(64, (shared_tiles + 1) / 2); ++p) {
    const int64_t len = (shared_tiles + p - 1) / p, items = int64_t(j.units) * at->kv_heads * p;
    const double t = double((items + slots - 1) / slots) * double(len + 3) * turn + double(p) * part;
    if (t < best) {
      best = t;
      how.cost = len;
    }
  }
  j.parts = int(build(j.list, u, j.per, at->kv_heads, slots, 1, how));
}

// Partial results of both sides of a join by rows.
struct RowParts {
  float4 *own_ml, *joint_ml;
  float *own, *joint;
  size_t bytes;
};

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

RowParts carve_row_parts(void* p, int64_t own_rows, int64_t joint_tiles, int dp) {
  Carve c{static_cast<char*>(p)};
  RowParts x{};
  x.own_ml = static_cast<float4*>(c.take(size_t(own_rows) * sizeof(float4)));
  x.joint_ml = static_cast<float4*>(c.take(size_t(joint_tiles) * 32 * sizeof(float4)));
  x.own = static_cast<float*>(c.take(size_t(own_rows) * size_t(dp) * 4));
  x.joint = static_cast<float*>(c.take(size_t(joint_tiles) * 32 * size_t(dp) * 4));
  x.bytes = c.used;
  return x;
}

size_t tile_bytes(const cgtp_attn_s* a) { return size_t(a->DP) * 32 * dtype_size(a->dtype); }

// Packed context: key row fragments, value column fragments, key biases.
struct Context {
  void *kf, *vf;
  float *bias, *norms;
  int32_t* flags;
  size_t bytes;
};
Context carve_context(const cgtp_attn_s* a, int64_t ktiles, void* p) {
  Carve c{static_cast<char*>(p)};
  const size_t n = size_t(ktiles) * size_t(a->kv_heads) * tile_bytes(a);
  Context x{};
  x.kf = c.take(n);
  x.vf = c.take(n);
  x.bias = static_cast<float*>(c.take(size_t(ktiles) * 32 * 4));
  x.norms = static_cast<float*>(c.take(size_t(ktiles) * size_t(a->kv_heads) * 4));
  x.flags = static_cast<int32_t*>(c.take(size_t(ktiles) * 4));
  x.bytes = c.used;
  return x;
}
Context carve_context(const cgtp_attn_batch_s* b, void* p) { return carve_context(b->attn, b->ktiles, p); }

struct Backward {
  char *kforms, *qforms;  // at strides of kbytes and qbytes
  size_t kbytes, qbytes;
  float *bias, *rows, *part_q, *part_k, *part_v;
  int32_t *k_bad, *q_bad;
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
  x.k_bad = static_cast<int32_t*>(c.take(b->causal ? size_t(b->ktiles) * g * 4 : 0));
  x.q_bad = static_cast<int32_t*>(c.take(b->causal ? size_t(b->qtiles) * g * 4 : 0));
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
  a->seq = dtype == CGTP_BF16 ? seq_kernels_bf16(a->DP) : seq_kernels_f32(a->DP);
  a->device = current_device();
  a->table.upload(table.data(), table.size() * sizeof(int4));
  return a.release();
}

cgtp_attn_batch_s* build_attn_batch(cgtp_attn_s* at, const cgtp_samples_s* q, const cgtp_samples_s* k, bool causal,
                                    int64_t shared) {
  if (q->S != k->S) throw Error{CGTP_ERR_INVALID_ARG, "attention: the two sides have different numbers of samples"};
  auto b = std::make_unique<cgtp_attn_batch_s>();
  b->attn = at;
  b->nq = q->rows;
  b->nk = shared + k->rows;
  b->device = current_device();
  if (b->nk > INT32_MAX - 64) throw Error{CGTP_ERR_UNSUPPORTED, "attention: context of more than 2^31 rows"};
  const Side qs = cut(q->ptr, at->G, 0, at->kv_heads), ks = cut(k->ptr, 1, shared, at->kv_heads);
  b->qtiles = int64_t(qs.tiles.size());
  b->ktiles = int64_t(ks.tiles.size());
  b->shared_tiles = (shared + 31) / 32;
  b->causal = causal;
  b->sequence = causal || shared > 0;
  // tokens and places (32 a tile) are compared in 32 bits
  if (causal && (b->nq > 1 << 30 || 32 * b->ktiles > 1 << 30))
    throw Error{CGTP_ERR_UNSUPPORTED, "attention: a causal batch of more than 2^30 rows"};
  b->qtile_mem.upload(qs.tiles.data(), qs.tiles.size() * sizeof(Tile));
  b->ktile_mem.upload(ks.tiles.data(), ks.tiles.size() * sizeof(Tile));
  const int g = at->kv_heads;
  const Sight sight{q->ptr, k->ptr, qs, ks, at->G, b->shared_tiles, causal};
  bool few = true;
  if (b->sequence) {
    std::vector<Reach> reach;
    for (size_t s = 0; s + 1 < qs.first.size(); ++s) {
      const int32_t n = qs.first[s + 1] - qs.first[s];
      few = few && n <= 1;
      reach.insert(reach.end(), size_t(n), sight.reach(s));
    }
    b->reach.upload(reach.data(), reach.size() * sizeof(Reach));
  }
  // samples with one query tile take the kernel whose waves share the queries,
  // those with enough rows the one of 64 rows a wave
  const int wide = wide_forward(at->DP, dtype_size(at->dtype)) ? kWideTiles : INT32_MAX;
  // workgroups at once: two a compute unit where registers and shared memory allow
  const int es = int(dtype_size(at->dtype)), two = 2 * kCus, one = kCus;
  const int slots = forward_slots(at);
  // Samples of a tile at most, which mostly hold less than 32 rows: their rows go against
  // the shared rows together where that saves enough products of tiles to pay for two more
  // launches (32-row tiles of heads of 128, us with and without: bf16 56,000 saved 47 and 60,
  // 14,300 saved 41 and 33; fp32 3600 saved 42 and 55, 900 saved 45 and 31).
  if (shared > 0 && few) {
    const int64_t saved = (b->qtiles - (b->nq * at->G + 31) / 32) * b->shared_tiles * g;
    if (saved * at->DP >= (es == 2 ? 3200000 : 450000)) build_joint(b->joint, at, b->nq, b->shared_tiles, false);
  }
  const bool joint = b->joint.per > 0;
  const auto forward = [&](WorkList& w, int per, int slots, int min_len, auto&& take) {
    std::vector<Unit> u;
    if (b->sequence)
      add_query_units(u, sight, per, 1, 0, joint, take);
    else
      add_units(u, qs, ks, 0, per, 1, {0}, take);
    build(w, u, per, g, slots, min_len, {joint, causal, false, b->sequence ? part_extra(at, per) : 5, 0, b->sequence});
  };
  // the items' tiles by a sample's: one, some, many
  int one_tile = 1, some = 4, many = 8;
  if (b->sequence && !joint) {
    // A kernel's launch costs some 10 us more than it does. Samples of one tile with short
    // contexts go along with those of more (us apart and together: samples of 1 - 60 rows 24
    // and 14 in bf16, 36 and 22 in fp32); small work of 64 rows a wave goes in 32, which
    // takes a twelfth longer, and little work beside it in 64.
    std::vector<Unit> u[3];
    add_query_units(u[0], sight, 1, 1, 0, false, [](int n) { return n == 1; });
    add_query_units(u[1], sight, 4, 1, 0, false, [&](int n) { return n > 1 && n < wide; });
    add_query_units(u[2], sight, 8, 1, 0, false, [&](int n) { return n >= wide; });
    double us[3] = {0, 0, 0};
    int64_t longest = 0;
    for (int i = 0; i < 3; ++i)
      for (const Unit& x : u[i]) {
        us[i] += double(x.tiles) * (x.b1 - x.b0) * g * at->DP * 4096 / (es == 2 ? 1e9 : 1.2e8);
        if (i == 0) longest = std::max<int64_t>(longest, x.b1 - x.b0);
      }
    if (!u[1].empty() && !u[2].empty()) {
      if (us[2] < 120) many = 4;
      else if (us[1] < 10) some = 8;
    }
    if (longest <= 16 && (!u[1].empty() || !u[2].empty())) one_tile = u[1].empty() ? many : some;
  }
  const auto kernel = [&](int n) { return n >= wide ? many : n > 1 ? some : n == 1 ? one_tile : 0; };
  forward(b->fwd, 4, slots, 4, [&](int n) { return kernel(n) == 4; });
  forward(b->wide, 8, two, 4, [&](int n) { return kernel(n) == 8; });
  forward(b->few, 1, slots, 8, [&](int n) { return kernel(n) == 1; });
  std::vector<Unit> u;
  const auto all = [](int) { return true; };
  if (b->sequence && at->seq.delta) {
    std::vector<int4> tiles;
    add_query_units(u, sight, 1, 1, 0, false, all);
    for (const Unit& x : u)
      if (x.b1 > x.b0 && x.b1 - x.b0 <= kFewKeyTiles) tiles.push_back({x.a0, x.b0, x.b1, 0});
    u.clear();
    b->few_keys = int(tiles.size());
    if (!tiles.empty()) b->few_keys_mem.upload(tiles.data(), tiles.size() * sizeof(int4));
  }
  const bool one_kind = one_pass(at->DP, dtype_size(at->dtype));
  const std::vector<int32_t> kinds = one_kind ? std::vector<int32_t>{kItemV} : std::vector<int32_t>{kItemV, kItemK};
  if (b->sequence) {
    add_query_units(u, sight, 4, 3, kItemQ, false, all);
    add_key_units(u, sight, 4, one_kind ? 4 : 3, kinds);
  } else {
    add_units(u, qs, ks, 0, 4, 3, {kItemQ}, all);
    add_units(u, ks, qs, 1, 4, one_kind ? 4 : 3, kinds, all);
  }
  build(b->bwd, u, 4, g, at->DP * es <= 384 ? two : one, 4, {false, causal, causal, 5, 0, b->sequence});
  return b.release();
}

namespace {
// Workgroups of a step that a compute unit holds at once, by their shared memory.
int64_t step_workgroups(int dp, size_t es) {
  const int64_t bytes = step_waves(dp, es) * 32 * int64_t(dp) * int64_t(es) * 5 / 2;
  return std::max<int64_t>(1, std::min<int64_t>(4, 160 * 1024 / bytes));
}
// Rows of partial results of a step against the caches (0: rows are final): StepCut.
int64_t step_part_rows(const cgtp_attn_cache_s* c) {
  if (c->whole || c->slots == 0) return 0;
  return (c->shares + c->qtiles) * c->attn->kv_heads * std::min(c->attn->G, 32);
}
}  // namespace

cgtp_attn_cache_s* build_attn_cache(cgtp_attn_s* at, int64_t slots, int64_t capacity, int64_t shared) {
  auto c = std::make_unique<cgtp_attn_cache_s>();
  c->attn = at;
  c->slots = slots;
  c->capacity = capacity;
  c->shared = shared;
  c->device = current_device();
  // (places are counted in 32 bits, beyond the end of a sequence's last turn)
  if (capacity > 1 << 30 || slots > INT32_MAX || shared > INT32_MAX - 64)
    throw Error{CGTP_ERR_UNSUPPORTED, "attention cache: more than 2^30 places a slot, or 2^31 slots or shared rows"};
  std::vector<int64_t> ptr;
  if (slots * at->G > INT32_MAX - 64) throw Error{CGTP_ERR_UNSUPPORTED, "attention: rows x heads beyond 2^31"};
  need_launch(slots * ((at->G + 31) / 32) * at->kv_heads);  // (before the lists are laid out, as the next)
  need_packing((shared + 31) / 32, at->kv_heads);
  for (int64_t s = 0; s <= slots; ++s) ptr.push_back(s);
  const Side qs = cut(ptr, at->G);
  c->qtiles = int64_t(qs.tiles.size());
  c->tiles_a_slot = (at->G + 31) / 32;
  const size_t es = dtype_size(at->dtype);
  const int waves = step_waves(at->DP, es);
  const int64_t tiles = (capacity + 31) / 32;
  if (c->qtiles * tiles > 1 << 30) throw Error{CGTP_ERR_UNSUPPORTED, "attention cache: more than 2^30 tiles of 32 places"};
  // Short caches of few slots: a workgroup a slot and head or two, in one launch (us so and shared
  // out: 8 slots of up to 64 places of heads of 72 in fp32 15 and 30; 32 slots of 256 of heads of
  // 128 in bf16 17 and 20, of 512 21 and 21; 200 slots of 128 38 and 36)
  const int64_t at_once = kCus * step_workgroups(at->DP, es);
  const int whole_waves = std::min(waves, tiles >= 4 ? 4 : tiles >= 2 ? 2 : 1);
  const int whole_heads = std::min(waves / whole_waves, at->kv_heads);
  c->whole = shared == 0 && tiles <= 2 * waves &&
             c->qtiles * ((at->kv_heads + whole_heads - 1) / whole_heads) <= at_once / 2;
  // neighbouring heads on the waves of a workgroup; where there are fewer heads than waves,
  // a head's waves take tiles in turn
  c->heads_a_group = c->whole ? whole_heads : std::min(waves, at->kv_heads);
  c->waves_a_head = c->whole ? whole_waves : waves / c->heads_a_group;
  c->bundles = (at->kv_heads + c->heads_a_group - 1) / c->heads_a_group;
  // as many workgroups as the device works on at once, each with two turns or more (64
  // sequences of up to 8000 tokens, heads of 128 in bf16: 124 us, with twice as many 130 us)
  c->shares = int(std::max<int64_t>(1, at_once / c->bundles));
  c->min_turns = 2;
  const int64_t workgroups = (std::max<int64_t>(c->qtiles, c->shares) + 7) / 8 * 8 * c->bundles;
  if (step_part_rows(c.get()) > INT32_MAX) throw Error{CGTP_ERR_UNSUPPORTED, "attention: too many partial rows"};
  // a row's pieces of the heads of a workgroup in their order in memory, of 16 bytes, 4
  // channels (where that is less) and one
  const int ve = 16 / int(es);
  const int widths[3] = {at->vec16 ? ve : 0, ve > 4 && at->quad ? 4 : 0, 1};
  for (int i = 0; i < 3; ++i) {
    if (widths[i] == 0) continue;
    std::vector<StepPiece> pieces;
    int d = 0;
    for (const RowBlock& k : at->krow.blocks) {
      const int cw = k.mul / at->kv_heads;
      for (int m = 0; m < k.nc; ++m, d += cw)
        for (int j = 0; j < c->heads_a_group; ++j)
          for (int e = 0; e < cw; e += widths[i]) pieces.push_back({k.off + m * k.mul + j * cw + e, cw, j, d + e});
    }
    c->width[i] = widths[i];
    c->pieces[i] = int(pieces.size());
    c->piece_mem[i].upload(pieces.data(), pieces.size() * sizeof(StepPiece));
  }
  std::vector<Join> joins;
  for (int64_t t = 0; t < c->qtiles; ++t)
    for (int hk = 0; hk < at->kv_heads; ++hk)
      joins.push_back({int32_t(t), hk, 0, 0, 1, 0, 0, 0});  // (parts: by the lengths)
  need_launch(int64_t(joins.size()));
  c->joins = int(joins.size());
  c->qtile_mem.upload(qs.tiles.data(), qs.tiles.size() * sizeof(Tile));
  c->join_mem.upload(joins.data(), joins.size() * sizeof(Join));
  if (shared > 0) {
    const Side ks = cut({0}, 1, shared);
    c->shared_tiles = int64_t(ks.tiles.size());
    c->shared_tile_mem.upload(ks.tiles.data(), ks.tiles.size() * sizeof(Tile));
    build_joint(c->joint, at, slots, c->shared_tiles, step_with_joint(at->DP, es));
  }
  need_launch(workgroups + (c->joint.list.items + 7) / 8 * 8);
  // short caches behind long shared rows: no more shares than the device holds beside those
  if (c->joint.per && c->qtiles * tiles <= 8 * int64_t(c->shares) * c->waves_a_head)
    c->shares = int(std::max<int64_t>(1, std::max(at_once / 4, at_once - c->joint.list.items) / c->bundles));
  return c.release();
}

size_t attn_context_bytes(const cgtp_attn_batch_s* b) { return carve_context(b, nullptr).bytes; }

size_t attn_forward_ws_bytes(const cgtp_attn_batch_s* b, bool packed) {
  if (b->joint.per)
    return carve_row_parts(nullptr, b->few.part_tiles[0] * 32, b->joint.list.part_tiles[0], b->attn->DP).bytes +
           (packed ? 0 : attn_context_bytes(b));
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

PackArgs context_pack(const cgtp_attn_s* a, const DevMem& tiles, int64_t ktiles, RowsIn k, RowsIn v,
                      const uint8_t* mask) {
  PackArgs p{};
  p.t[0].src = k.p;
  p.t[0].ld = k.ld;
  p.t[0].vec = vec_rows(a, k.p, k.ld);
  p.t[1].src = v.p;
  p.t[1].ld = v.ld;
  p.t[1].vec = vec_rows(a, v.p, v.ld);
  p.tiles = tiles.as<Tile>();
  p.ntiles = int(ktiles);
  p.table = a->table.as<int4>();
  p.size = a->D;
  p.mask = mask;
  p.heads = a->heads;
  p.groups = a->kv_heads;
  return p;
}

// Packs the context's keys and values for the forward.
void pack_forward(const cgtp_attn_s* a, const DevMem& tiles, int64_t ktiles, RowsIn k, RowsIn v, const uint8_t* mask,
                  const Context& c, hipStream_t s) {
  PackArgs p = context_pack(a, tiles, ktiles, k, v, mask);
  p.t[0].row_frags = c.kf;
  p.bias = c.bias;
  p.flags = c.flags;
  p.norms = c.norms;
  p.t[1].col_frags = c.vf;
  a->k.pack(p, s);
  CGTP_CHECK_HIP(hipGetLastError());
}

FwdArgs forward_args(const cgtp_attn_s* a, RowsIn q, double scale, void* out, float* lse) {
  FwdArgs f{};
  f.table = a->table.as<int4>();
  f.q = q.p;
  f.ldq = q.ld;
  f.q_vec = vec_rows(a, q.p, q.ld);
  f.out = out;
  f.ldo = a->qrow.dim;
  f.out_quad = quad_rows(a, out);
  f.lse = lse;
  // a zero scale stays a small positive one: every score is then 0 all the same
  f.scale2 = std::max(float(std::fabs(scale) * 1.4426950408889634), 1e-37f);
  f.q_sign = scale < 0.0 ? (a->dtype == CGTP_BF16 ? 0x80008000u : 0x80000000u) : 0u;
  f.G = a->G;
  f.heads = a->heads;
  f.groups = a->kv_heads;
  return f;
}

void use_context(FwdArgs& f, const Context& c) {
  f.kf = c.kf;
  f.vf = c.vf;
  f.bias = c.bias;
  f.flags = c.flags;
  f.norms = c.norms;
}

// All rows against the shared ones, as parts.
void joint_launch(const cgtp_attn_s* a, const JointPlan& j, FwdArgs f, const RowParts& w, hipStream_t s) {
  f.qtiles = j.tiles.as<Tile>();
  f.items = j.list.item_mem.as<Item>();
  f.part = w.joint;
  f.part_ml = w.joint_ml;
  a->k.fwd(f, j.list.items, j.per, s);
  CGTP_CHECK_HIP(hipGetLastError());
}

StepCut step_cut(const cgtp_attn_cache_s* c, const int32_t* lengths, int32_t* before) {
  return {lengths,         int(c->slots), int(c->capacity), c->tiles_a_slot,
          c->waves_a_head, c->shares,     c->min_turns,     before};
}

void rows_join_launch(const cgtp_attn_s* a, const JointPlan& j, const FwdArgs& own, const RowParts& w, int joins,
                      const StepCut& cut, hipStream_t s) {
  const RowsJoinArgs r{own, w.joint, w.joint_ml, j.units, j.per, j.per ? j.parts : 0, cut};
  a->seq.rows_join(r, joins, s);
  CGTP_CHECK_HIP(hipGetLastError());
}

}  // namespace

void attn_pack_launch(const cgtp_attn_batch_s* b, RowsIn k, RowsIn v, const uint8_t* mask, void* context,
                      hipStream_t s) {
  if (b->ktiles) pack_forward(b->attn, b->ktile_mem, b->ktiles, k, v, mask, carve_context(b, context), s);
}

void attn_forward_launch(const cgtp_attn_batch_s* b, RowsIn q, const void* context, double scale, void* out,
                         float* lse, void* ws, hipStream_t s) {
  const cgtp_attn_s* a = b->attn;
  FwdArgs f = forward_args(a, q, scale, out, lse);
  use_context(f, carve_context(b, const_cast<void*>(context)));
  f.qtiles = b->qtile_mem.as<Tile>();
  f.reach = b->reach.as<Reach>();
  f.shared = int(b->shared_tiles);
  f.causal = b->causal;
  if (b->joint.per) {
    const RowParts w = carve_row_parts(ws, b->few.part_tiles[0] * 32, b->joint.list.part_tiles[0], a->DP);
    joint_launch(a, b->joint, f, w, s);
    f.items = b->few.item_mem.as<Item>();
    f.joins = b->few.join_mem[0].as<Join>();
    f.part = w.own;
    f.part_ml = w.own_ml;
    a->seq.fwd(f, b->few.items, 1, s);
    CGTP_CHECK_HIP(hipGetLastError());
    rows_join_launch(a, b->joint, f, w, b->few.joins[0], {}, s);
    return;
  }
  f.part_ml = static_cast<float4*>(ws);
  f.part = reinterpret_cast<float*>(f.part_ml + size_t(fwd_part_tiles(b)) * 32);
  // the lists share the partial buffers: each is joined before the next starts
  for (const int tiles : {8, 4, 1}) {
    const WorkList& w = tiles == 8 ? b->wide : tiles == 4 ? b->fwd : b->few;
    if (w.items == 0) continue;
    f.items = w.item_mem.as<Item>();
    f.joins = w.join_mem[0].as<Join>();
    (b->sequence ? a->seq.fwd : a->k.fwd)(f, w.items, tiles, s);
    CGTP_CHECK_HIP(hipGetLastError());
    if (w.joins[0]) {
      a->k.fwd_join(f, w.joins[0], s);
      CGTP_CHECK_HIP(hipGetLastError());
    }
  }
}

size_t attn_cache_shared_bytes(const cgtp_attn_cache_s* c) {
  return carve_context(c->attn, c->shared_tiles, nullptr).bytes;
}

namespace {
RowParts carve_step(const cgtp_attn_cache_s* c, void* ws) {
  return carve_row_parts(ws, step_part_rows(c), c->joint.list.part_tiles[0], c->attn->DP);
}
}  // namespace

namespace {
// StepCut::before, behind the partial results
bool step_sums(const cgtp_attn_cache_s* c) { return !c->whole && c->slots >= kStepSumSlots; }
int32_t* step_before(const cgtp_attn_cache_s* c, void* ws) {
  return step_sums(c) ? reinterpret_cast<int32_t*>(static_cast<char*>(ws) + carve_step(c, nullptr).bytes) : nullptr;
}
}  // namespace

size_t attn_step_ws_bytes(const cgtp_attn_cache_s* c) {
  return carve_step(c, nullptr).bytes + (step_sums(c) ? size_t(c->slots + 1) * 4 : 0);
}

void attn_share_launch(const cgtp_attn_cache_s* c, RowsIn k, RowsIn v, const uint8_t* mask, void* context,
                       hipStream_t s) {
  if (c->shared_tiles)
    pack_forward(c->attn, c->shared_tile_mem, c->shared_tiles, k, v, mask,
                 carve_context(c->attn, c->shared_tiles, context), s);
}

void attn_step_launch(const cgtp_attn_cache_s* c, RowsIn q, RowsIn k, RowsIn v, void* k_cache, void* v_cache,
                      const int32_t* lengths, const void* context, double scale, void* out, float* lse, void* ws,
                      hipStream_t s) {
  const cgtp_attn_s* a = c->attn;
  const RowParts w = carve_step(c, ws);
  FwdArgs f = forward_args(a, q, scale, out, lse);
  FwdArgs shared = f;
  if (c->joint.per) {
    use_context(shared, carve_context(a, c->shared_tiles, const_cast<void*>(context)));
    shared.qtiles = c->joint.tiles.as<Tile>();
    shared.items = c->joint.list.item_mem.as<Item>();
    shared.part = w.joint;
    shared.part_ml = w.joint_ml;
  }
  f.qtiles = c->qtile_mem.as<Tile>();
  f.joins = c->join_mem.as<Join>();
  f.part = w.own;
  f.part_ml = w.own_ml;
  StepArgs x{};
  x.f = f;
  x.k_new = k.p;
  x.v_new = v.p;
  x.ldk = k.ld;
  x.ldv = v.ld;
  x.k_cache = k_cache;
  x.v_cache = v_cache;
  x.dim = a->krow.dim;
  x.cut = step_cut(c, lengths, step_before(c, ws));
  if (x.cut.before) {
    a->seq.step_sums(x.cut, s);
    CGTP_CHECK_HIP(hipGetLastError());
  }
  x.size = a->D;
  x.heads_a_group = c->heads_a_group;
  x.bundles = c->bundles;
  x.whole = c->whole;
  x.joined = c->joint.per > 0;
  // the widest pieces that the caches' rows are made of, by their alignment
  for (int i = 2; i >= 0; --i) {
    const size_t bytes = size_t(c->width[i]) * dtype_size(a->dtype);
    if (c->width[i] == 0 || !aligned(k_cache, bytes) || !aligned(v_cache, bytes) ||
        size_t(x.dim) * dtype_size(a->dtype) % bytes != 0)
      continue;
    x.width = c->width[i];
    x.pieces = c->pieces[i];
    x.piece = c->piece_mem[i].as<StepPiece>();
  }
  if (c->joint.per) {
    if (step_with_joint(a->DP, dtype_size(a->dtype)) && x.width * dtype_size(a->dtype) == 16) {
      x.joint = shared;
      x.joint_items = c->joint.list.items;
      x.joint_blocks = (x.joint_items + 7) / 8 * 8;
    } else {
      a->k.fwd(shared, c->joint.list.items, c->joint.per, s);
      CGTP_CHECK_HIP(hipGetLastError());
    }
  }
  a->seq.step(x, s);
  CGTP_CHECK_HIP(hipGetLastError());
  if (!x.whole) rows_join_launch(a, c->joint, f, w, c->joins, x.cut, s);
}

void attn_backward_launch(const cgtp_attn_batch_s* b, RowsIn q, RowsIn k, RowsIn v, const uint8_t* mask, double scale,
                          const void* out, const float* lse, RowsIn g, void* dq, void* dk, void* dv, void* ws,
                          hipStream_t s) {
  const cgtp_attn_s* a = b->attn;
  const Backward w = carve_backward(b, ws);
  if (b->ktiles) {
    PackArgs p = context_pack(a, b->ktile_mem, b->ktiles, k, v, mask);
    p.t[0].row_frags = w.kforms + kKRows * w.kbytes;
    p.t[0].col_frags = dq ? w.kforms + kKCols * w.kbytes : nullptr;
    p.bias = w.bias;
    p.t[1].row_frags = w.kforms + kVRows * w.kbytes;
    p.bad = w.k_bad;
    (b->causal ? a->seq.pack : a->k.pack)(p, s);
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
    p.bad = w.q_bad;
    (b->causal ? a->seq.pack : a->k.pack)(p, s);
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
  x.reach = b->reach.as<Reach>();
  x.shared = int(b->shared_tiles);
  x.causal = b->causal;
  x.k_bad = w.k_bad;
  x.q_bad = w.q_bad;
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
  if (b->few_keys && (dq || dk)) {
    a->seq.delta(x, b->few_keys_mem.as<int4>(), b->few_keys, w.rows, s);
    CGTP_CHECK_HIP(hipGetLastError());
  }
  x.items = l.item_mem.as<Item>();
  (b->sequence ? a->seq.bwd : a->k.bwd)(x, l.items, s);
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
