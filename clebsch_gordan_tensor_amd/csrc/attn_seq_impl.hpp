// Attention along sequences: one token's step on caches of irreps rows, and the join of
// results against rows that samples share with those against their own (kernels
// templated as attn_impl.hpp's; instantiated in inst/attn_seq_*.hip).
#pragma once

#include "attn_impl.hpp"

namespace cgtp {
namespace attn {

// ---------------------------------------------------------------------- step
//
// One query token a slot against the slot's cached rows and the new one, which is put
// into the cache by the workgroups that take its place. A wave takes one tile of query
// rows (the heads that share a context head) and a part of the places, 32 keys a turn:
// S^T = K Q^T, O^T += V^T P^T as in fwd_few_kernel, the values turned from rows to columns
// by way of shared memory. The rows stay as the caller has them: no packing, and a cache
// can be read, copied or cut with ordinary tensor operations.
//
// Bound: the cached rows' bytes. A head's channels are short runs of a row (16 bytes for
// 32 channels over 4 heads in bf16), so a workgroup takes neighbouring heads, whose runs lie
// in the same cache lines, and the other heads' workgroups follow on the same die
// (workgroup index modulo 8).

// W channels of one row in registers.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <typename T, int W>
struct Piece {
  static constexpr int kBytes = W * int(sizeof(T)), kWords = (kBytes + 3) / 4;
  using V = std::conditional_t<kBytes == 16, u32x4, std::conditional_t<kBytes == 8, u32x2, uint32_t>>;
  using M = std::conditional_t<kBytes == 2, uint16_t, V>;  // in memory
  V d;
  __device__ __forceinline__ void load(const char* p) { d = V(*reinterpret_cast<const M*>(p)); }
  __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<M*>(p) = M(d); }
  __device__ __forceinline__ void clear_unless(bool keep) { d = keep ? d : V(0); }
  __device__ __forceinline__ uint32_t word(int i) const {
    if constexpr (kWords == 1) return d;
    else return d[i];
  }
};

// The values of a tile by columns (a head's elements) of 32 keys, as operands: quads of 4
// keys turned from rows in registers.
template <typename T>
struct Columns;
template <>
struct Columns<bf16> {
  static constexpr int kStride = 80;  // bytes a column: 32 keys and 16 against bank conflicts
  // Byte of quad q in column d: column fragment f, half h hold quads 4 f + h and
  // 4 f + 2 + h next to each other, as 16 bytes whose place turns with d / 16 (else the
  // columns that a wave writes at once would start at two banks: 174 us, with it 142 us).
  static __device__ __forceinline__ int at(int d, int q) {
    return d * kStride + ((q / 4 * 2 + q % 2) ^ (d / 16 & 3)) * 16 + q / 2 % 2 * 8;
  }
  static __device__ __forceinline__ int frag(int d, int f, int h) {
    return d * kStride + ((2 * f + h) ^ (d / 16 & 3)) * 16;
  }
  template <int W>
  static __device__ __forceinline__ void turn(const Piece<bf16, W> (&r)[4], char* column) {
#pragma unroll
    for (int c = 0; c < Piece<bf16, W>::kWords; ++c) {
      uint2 v;
      v.x = __builtin_amdgcn_perm(r[1].word(c), r[0].word(c), 0x05040100);
      v.y = __builtin_amdgcn_perm(r[3].word(c), r[2].word(c), 0x05040100);
      *reinterpret_cast<uint2*>(column + 2 * c * kStride) = v;
      if constexpr (W > 1) {
        v.x = __builtin_amdgcn_perm(r[1].word(c), r[0].word(c), 0x07060302);
        v.y = __builtin_amdgcn_perm(r[3].word(c), r[2].word(c), 0x07060302);
        *reinterpret_cast<uint2*>(column + (2 * c + 1) * kStride) = v;
      }
    }
  }
};
template <>
struct Columns<float> {
  static constexpr int kStride = 144;
  static __device__ __forceinline__ int at(int d, int q) { return d * kStride + (q ^ (d / 16 & 7)) * 16; }
  static __device__ __forceinline__ int frag(int d, int f, int h) { return at(d, 2 * f + h); }
  template <int W>
  static __device__ __forceinline__ void turn(const Piece<float, W> (&r)[4], char* column) {
#pragma unroll
    for (int c = 0; c < W; ++c)
      *reinterpret_cast<u32x4*>(column + c * kStride) = u32x4{r[0].word(c), r[1].word(c), r[2].word(c), r[3].word(c)};
  }
};

// A barrier for what is in shared memory: loads from memory stay on their way.
__device__ __forceinline__ void turn_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// Orders a wave's own writes and reads of shared memory.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = lane_id();
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const int o = __builtin_amdgcn_ds_bpermute((lane - off) << 2, v);
    v += lane >= off ? o : 0;
  }
  return v;
}
// Turns of one tile of rows of a slot of length `len`.
__device__ __forceinline__ int step_turns(const StepCut& c, int len) {
  return len >= 0 && len < c.capacity ? (len / 32 + c.waves_a_head) / c.waves_a_head : 0;
}
// The turns of a slot's tiles, for every slot one after another.
struct StepTurns {
  int mine, upto, each;  // this lane's run of `each` slots: its turns, and those up to its end
  int total;
};
__device__ __forceinline__ StepTurns step_sum(const StepCut& c) {
  StepTurns s;
  if (c.before) {
    s.mine = s.upto = s.each = 0;
    s.total = ldc(c.before + c.slots);
    return s;
  }
  s.each = (c.slots + 63) / 64;
  s.mine = 0;
  const int first = lane_id() * s.each, end = min(first + s.each, c.slots);
#pragma unroll 4
  for (int i = first; i < end; ++i) s.mine += step_turns(c, c.lengths[i]) * c.tiles_a_slot;
  s.upto = wave_scan(s.mine);
  s.total = __builtin_amdgcn_readlane(s.upto, 63);
  return s;
}
// Turns of a workgroup's stretch.
__device__ __forceinline__ int step_share(const StepCut& c, int total) {
  return max(c.min_turns, (total + c.shares - 1) / c.shares);
}
// Turns before slot `slot`.
__device__ __forceinline__ int step_before(const StepCut& c, const StepTurns& s, int slot) {
  if (c.before) return ldc(c.before + slot);
  const int run = slot / s.each;
  int n = __builtin_amdgcn_readlane(s.upto - s.mine, run);
  for (int i = run * s.each; i < slot; ++i) n += step_turns(c, ldc(c.lengths + i)) * c.tiles_a_slot;
  return n;
}
// The slot that turn `at` (below the total) belongs to, and its first turn.
__device__ __forceinline__ int2 step_find(const StepCut& c, const StepTurns& s, int at) {
  if (c.before) {
    // the last slot that begins at or before it
    int lo = 0, hi = c.slots;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      (ldc(c.before + mid) <= at ? lo : hi) = mid;
    }
    return make_int2(lo, ldc(c.before + lo));
  }
  const int run = __builtin_ctzll(__ballot(s.upto > at));
  int slot = run * s.each, n = __builtin_amdgcn_readlane(s.upto - s.mine, run);
  while (true) {
    const int turns = step_turns(c, ldc(c.lengths + slot)) * c.tiles_a_slot;
    if (n + turns > at) return make_int2(slot, n);
    n += turns;
    ++slot;
  }
}

// StepCut::before, by one workgroup.
constexpr int kSumThreads = 1024;
static __global__ __launch_bounds__(kSumThreads) void step_sums_kernel(StepCut c) {
  __shared__ int waves[kSumThreads / 64];
  const int tid = int(threadIdx.x), each = (c.slots + kSumThreads - 1) / kSumThreads;
  const int first = min(tid * each, c.slots), end = min(first + each, c.slots);
  int mine = 0;
  for (int i = first; i < end; ++i) mine += step_turns(c, c.lengths[i]) * c.tiles_a_slot;
  const int upto = wave_scan(mine);
  if (tid % 64 == 63) waves[tid / 64] = upto;
  __syncthreads();
  int n = upto - mine;
  for (int k = 0; k < tid / 64; ++k) n += waves[k];
  for (int i = first; i < end; ++i) {
    c.before[i] = n;
    n += step_turns(c, c.lengths[i]) * c.tiles_a_slot;
  }
  if (tid == kSumThreads - 1) c.before[c.slots] = n;
}

// The part of workgroup `index` and tile of rows qt.
__device__ __forceinline__ int step_part(const StepCut& c, int hk, int index, int qt) {
  return hk * (c.shares + c.slots * c.tiles_a_slot) + index + qt;
}

// What a workgroup does next: turns a .. b - 1 of tile of rows qt.
struct StepWork {
  int hk;   // this wave's context head
  bool on;  // (the last workgroup of a row may have fewer heads than waves)
  int index, bundle, at, end;
  int slot, before;  // the slot of turn `at` and the turns before it
  int qt, len, t0, t1;  // key tiles t0 .. t1 - 1
  Item it;
};
// False: the workgroup has nothing to do.
__device__ __forceinline__ bool step_begin(const StepArgs& a, int block, int wave, StepWork& w) {
  const int turn = block / 8;
  w.bundle = turn % a.bundles;
  w.index = turn / a.bundles * 8 + block % 8;
  const int j = wave / a.cut.waves_a_head;
  w.hk = w.bundle * a.heads_a_group + j;
  w.on = j < a.heads_a_group && w.hk < a.f.groups;
  if (a.whole) {
    w.at = 0;
    w.end = 1;
    return w.index < a.cut.slots * a.cut.tiles_a_slot;
  }
  if (w.index >= a.cut.shares) return false;
  const StepTurns s = step_sum(a.cut);
  const int share = step_share(a.cut, s.total);
  // (a product of the shares' number and length may pass 32 bits, but not by much)
  const int64_t at = int64_t(w.index) * share;
  if (at >= s.total) return false;
  w.at = int(at);
  w.end = min(w.at + share, s.total);
  const int2 f = step_find(a.cut, s, w.at);
  w.slot = f.x;
  w.before = f.y;
  return true;
}
// The next stretch of one tile of rows; false at the end.
__device__ __forceinline__ bool step_next(const StepArgs& a, int wave, StepWork& w) {
  if (w.at >= w.end) return false;
  const int wph = a.cut.waves_a_head;
  if (a.whole) {
    w.at = 1;
    w.qt = w.index;
    w.slot = w.qt / a.cut.tiles_a_slot;
    w.len = ldc(a.cut.lengths + w.slot);
    const int turns = step_turns(a.cut, w.len);
    w.t0 = 0;
    w.t1 = turns > 0 ? w.len / 32 + 1 : 0;
    w.it = {w.qt, 1, w.t0, w.t1, w.hk, -1, 1, 0};
    return true;
  }
  int turns;
  while (true) {
    w.len = ldc(a.cut.lengths + w.slot);
    turns = step_turns(a.cut, w.len);
    if (w.at < w.before + turns * a.cut.tiles_a_slot) break;
    w.before += turns * a.cut.tiles_a_slot;
    ++w.slot;
  }
  const int within = w.at - w.before, tile = within / turns, first = within % turns;
  const int last = min(turns, first + w.end - w.at);
  w.at += last - first;
  w.qt = w.slot * a.cut.tiles_a_slot + tile;
  w.t0 = first * wph;
  w.t1 = min(last * wph, w.len / 32 + 1);
  const bool alone = first == 0 && last == turns && !a.joined;
  w.it = {w.qt, 1, w.t0, w.t1, w.hk, alone ? -1 : step_part(a.cut, w.hk, w.index, w.qt), 1, 0};
  return true;
}

// The new rows' elements of the wave's head into the caches, and what else `also` does
// with each of them (element d of the head).
template <typename T, typename F>
__device__ __forceinline__ void take_new(const StepArgs& a, const StepWork& w, F&& also) {
  const T* const k = static_cast<const T*>(a.k_new) + w.slot * a.ldk;
  const T* const v = static_cast<const T*>(a.v_new) + w.slot * a.ldv;
  const int64_t at = (int64_t(w.slot) * a.cut.capacity + w.len) * a.dim;
  const bool store = w.qt % a.cut.tiles_a_slot == 0;
  for (int d = lane_id(); d < a.size; d += 64) {
    const int64_t i = elem(a.f.table[d], false, w.hk);
    const T x = k[i], y = v[i];
    also(d, x, y);
    if (store) {
      static_cast<T*>(a.k_cache)[at + i] = x;
      static_cast<T*>(a.v_cache)[at + i] = y;
    }
  }
}

// Softmax and O^T of a tile: scores sc, values by columns in shared memory.
template <typename T, int DP>
__device__ __forceinline__ void step_weigh(const StepArgs& a, int t, int len, Running<DP / 32>& st, f32x16& sc, float& e,
                                           bool exact, typename Op<T>::Frag (&w)[16 / Op<T>::VE]) {
  if (32 * t + 31 > len) hide_later(sc, t, len + 1, lane_id() / 32);
  raise_reference(st, top_score(sc, a.f.scale2), e, exact);
  weigh<T, true>(st, sc, a.f.scale2, 0.0f, e, exact, w);
}
template <typename T, int DP>
__device__ __forceinline__ void step_values(const char* columns, int lane, Running<DP / 32>& st,
                                            const typename Op<T>::Frag (&w)[16 / Op<T>::VE]) {
  using D = Dims<T, DP>;
#pragma unroll
  for (int d = 0; d < D::DT; ++d)
#pragma unroll
    for (int f = 0; f < D::FR; ++f) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(columns + Columns<T>::frag(32 * d + lane % 32, f, lane / 32));
      st.o[d] = Op<T>::mma(as_frag<typename Op<T>::Frag>(x), w[f], st.o[d]);
    }
}

// Shared memory of a step: for every wave its rows of keys and its columns of values, with
// paddings against bank conflicts.
template <typename T, int DP>
struct StepShared {
  static constexpr int kWaves = step_waves(DP, sizeof(T));
  static constexpr int kRow = DP * int(sizeof(T)) + 16, kKeys = 32 * kRow, kPlace = kKeys + DP * Columns<T>::kStride + 64;
  char place[kWaves][kPlace];
  float ml[kWaves][3][64];
  // two workgroups a compute unit, where its 160 KB hold this twice
  static constexpr int kWavesASimd = kWaves * (kPlace + 768) <= 80 * 1024 ? few_waves(DP, sizeof(T)) : 1;
};
// Whether the registers hold the next turn's rows.
constexpr bool step_ahead(int dp, size_t size) { return dp * int(size) <= 512 && dp <= 192; }

// The waves of a head joined in the first of them, in a fixed order, by way of their places.
template <typename T, int DP>
__device__ __forceinline__ void join_waves(StepShared<T, DP>& sh, int wave, int wph, Running<DP / 32>& st, float& e) {
  const int lane = lane_id(), head = wave / wph * wph;
  sh.ml[wave][0][lane] = st.m;
  turn_lds();
  float m = -INFINITY;
  for (int k = 0; k < wph; ++k) m = fmaxf(m, sh.ml[min(head + k, StepShared<T, DP>::kWaves - 1)][0][lane]);
  const float f = m == -INFINITY ? 1.0f : exp2_fast(st.m - m);
  st.m = m;
  st.l *= f;
  e *= f;
  sh.ml[wave][1][lane] = st.l;
  sh.ml[wave][2][lane] = e;
#pragma unroll
  for (int d = 0; d < DP / 32; ++d) {
    st.o[d] *= f;
    f32x4* const box = reinterpret_cast<f32x4*>(sh.place[wave]);
    if (wave != head)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        box[b * 64 + lane] = f32x4{st.o[d][4 * b], st.o[d][4 * b + 1], st.o[d][4 * b + 2], st.o[d][4 * b + 3]};
    turn_lds();
    if (wave == head)
      for (int k = 1; k < wph; ++k) {
        const f32x4* const from = reinterpret_cast<const f32x4*>(sh.place[head + k]);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const f32x4 x = from[b * 64 + lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) st.o[d][4 * b + i] += x[i];
        }
      }
    turn_lds();
  }
  if (wave == head)
    for (int k = 1; k < wph; ++k) {
      st.l += sh.ml[head + k][1][lane];
      e += sh.ml[head + k][2][lane];
    }
}

// The workgroup reads the rows of its heads in their order in memory, quads of 4 keys x
// W channels a lane, a turn ahead in registers (reading every head's pieces straight as
// operands took twice as long: each load then touches 64 cache lines), and lays them out in
// shared memory: keys by rows, values by columns, each wave's tile in a place of its own.
// W: 16 bytes, 8 or one channel, by the heads' sizes and the tensors' alignment.
// Measured: 64 sequences of 1000 - 8000 tokens, heads of 128, bf16: 116 us = 5.1 TB/s.
template <typename T, int DP, int W>
__device__ __forceinline__ void step_body(const StepArgs& a, int block, StepShared<T, DP>& sh) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  using C = Columns<T>;
  using S = StepShared<T, DP>;
  constexpr int WAVES = S::kWaves, THREADS = 64 * WAVES, PER = (DP / W + 7) / 8;
  constexpr bool kSingle = W == 1;  // too many quads a thread to keep their places
  StepWork w;
  const int tid = int(threadIdx.x), wave = wave_id(), lane = lane_id(), n = lane % 32, h = lane / 32;
  if (!step_begin(a, block, wave, w)) return;
  const int wph = a.cut.waves_a_head;
  const int hk0 = w.hk - wave / wph, heads = min(a.heads_a_group, a.f.groups - hk0);
  // quads of this thread: one piece of four keys each (threads without one, and those of
  // heads that the last workgroup of a row does not have, repeat another's)
  const int row_bytes = int(a.dim * int64_t(sizeof(T)));
  struct Spot {
    int key, row_at, column_at;
    uint32_t off;  // bytes from the row's start
  };
  const auto spot = [&](int i) {
    i %= 8 * wph * a.pieces;
    const int quad = i / a.pieces;
    StepPiece p = a.piece[i % a.pieces];
    if (p.j >= heads) p = a.piece[0];
    const int place = (p.j * wph + quad / 8) * S::kPlace;
    return Spot{4 * quad, place + quad % 8 * 4 * S::kRow + p.d * int(sizeof(T)), place + S::kKeys + C::at(p.d, quad % 8),
                uint32_t(p.off + hk0 * p.cw) * uint32_t(sizeof(T))};
  };
  char* const mem = &sh.place[0][0];
  // Quad of the turn from tile t on. Places behind the sequence's end are read as well
  // (they are hidden), but none behind the caches' end.
  const auto load = [&](const void* cache, int t, const Spot& p, Piece<T, W> (&x)[4]) {
    const int64_t row = int64_t(w.slot) * a.cut.capacity + int64_t(t) * 32;
    const char* const base = static_cast<const char*>(cache) + row * row_bytes;
    const int rows = int(min(int64_t(a.cut.slots) * a.cut.capacity - row, int64_t(32 * WAVES)));
#pragma unroll
    for (int r = 0; r < 4; ++r)
      x[r].load(base + (p.off + (p.key + r < rows ? uint32_t(p.key + r) * uint32_t(row_bytes) : 0u)));
  };
  const auto put_keys = [&](const Spot& p, const Piece<T, W> (&x)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r].store(mem + p.row_at + r * S::kRow);
  };
  const auto put_values = [&](int t, const Spot& p, Piece<T, W> (&x)[4]) {
    // weight 0 times what a place from the end on holds would be NaN for infinities
    if (32 * (t + wph) > w.len)
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r].clear_unless(32 * t + p.key + r < w.len);
    C::turn(x, mem + p.column_at);
  };
  Spot spots[kSingle ? 1 : PER];
  if constexpr (!kSingle)
#pragma unroll
    for (int g = 0; g < PER; ++g) spots[g] = spot(tid + THREADS * g);
  // the widest heads leave no registers for the next turn's rows
  constexpr bool kAhead = !kSingle && step_ahead(DP, sizeof(T)) && (W == D::VE || DP <= 96);
  const bool exact = sizeof(T) == 2 && a.f.lse != nullptr;
  while (step_next(a, wave, w)) {
    Piece<T, W> k[kAhead ? PER : 1][4], v[kAhead ? PER : 1][4];
    const auto load_all = [&](const void* cache, int t, Piece<T, W> (&x)[kAhead ? PER : 1][4]) {
#pragma unroll
      for (int g = 0; g < (kAhead ? PER : 0); ++g) load(cache, t, spots[g], x[g]);
    };
    if (kAhead && w.t0 < w.t1) {
      load_all(a.k_cache, w.t0, k);
      load_all(a.v_cache, w.t0, v);
    }
    // (keys' places beyond the head meet zeros of the queries, and must not be NaN; the
    // join of waves writes there)
    if (a.size < DP)
      for (int i = lane; i < 32 * (DP - a.size); i += 64)
        *reinterpret_cast<T*>(&sh.place[wave][i % 32 * S::kRow + (a.size + i / 32) * int(sizeof(T))]) = T{};
    const Tile tl = ldc(a.f.qtiles + w.qt);
    Frag q[D::KSTEPS];
    load_queries<T, DP>(a.f, tl, w.on ? w.hk : 0, lane, q);
    Running<D::DT> st;
    float e = 0.0f;
#pragma unroll
    for (int d = 0; d < D::DT; ++d) st.o[d] = zero16();
    for (int t = w.t0; t < w.t1; t += wph) {
      const int mine = t + wave % wph;
      if constexpr (kAhead) {
        // (each tensor's registers are on their way again as soon as they are written out, so
        // that the reads of memory do not run dry)
        const int next = t + wph < w.t1 ? t + wph : t;
#pragma unroll
        for (int g = 0; g < PER; ++g) put_keys(spots[g], k[g]);
        load_all(a.k_cache, next, k);
#pragma unroll
        for (int g = 0; g < PER; ++g) put_values(t, spots[g], v[g]);
        load_all(a.v_cache, next, v);
      } else if constexpr (!kSingle) {
        // some quads of both tensors at a time
        constexpr int SOME = DP * int(sizeof(T)) > 768 ? 2 : 4;
#pragma unroll
        for (int g0 = 0; g0 < PER; g0 += SOME) {
          Piece<T, W> x[SOME][4];
#pragma unroll
          for (int tensor = 0; tensor < 2; ++tensor) {
#pragma unroll
            for (int g = g0; g < min(g0 + SOME, PER); ++g) load(tensor ? a.v_cache : a.k_cache, t, spots[g], x[g - g0]);
#pragma unroll
            for (int g = g0; g < min(g0 + SOME, PER); ++g) {
              if (tensor) put_values(t, spots[g], x[g - g0]);
              else put_keys(spots[g], x[g - g0]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      } else {
        const int count = 8 * wph * a.pieces;
#pragma unroll 4
        for (int i = tid; i < count; i += THREADS) {
          const Spot p = spot(i);
          Piece<T, W> x[4], y[4];
          load(a.k_cache, t, p, x);
          load(a.v_cache, t, p, y);
          put_keys(p, x);
          put_values(t, p, y);
        }
      }
      turn_lds();
      if (w.on && mine < w.t1) {
        if (mine == w.len / 32) {
          const int r = w.len % 32;
          take_new<T>(a, w, [&](int d, T x, T y) {
            *reinterpret_cast<T*>(&sh.place[wave][r * S::kRow + d * int(sizeof(T))]) = x;
            *reinterpret_cast<T*>(&sh.place[wave][S::kKeys + C::at(d, r / 4) + r % 4 * int(sizeof(T))]) = y;
          });
          wave_fence();
        }
        f32x16 sc = zero16();
#pragma unroll
        for (int u = 0; u < D::KSTEPS; ++u) {
          // (products of fp32 take eight times as long: none with padding alone)
          if (sizeof(T) == 4 && 2 * D::VE * u >= a.size) break;
          const u32x4 x = *reinterpret_cast<const u32x4*>(&sh.place[wave][n * S::kRow + (2 * u + h) * 16]);
          sc = Op<T>::mma(as_frag<Frag>(x), q[u], sc);
        }
        Frag p[D::FR];
        step_weigh<T, DP>(a, mine, w.len, st, sc, e, exact, p);
        step_values<T, DP>(&sh.place[wave][S::kKeys], lane, st, p);
      }
      turn_lds();
    }
    if (wph > 1) join_waves<T, DP>(sh, wave, wph, st, e);
    if (w.on && wave % wph == 0) finish<T, DP>(a.f, w.it, tl, 0, st, e, min(a.f.G, 32));
  }
}

template <typename T, int DP, int W>
__global__ __launch_bounds__(64 * step_waves(DP, sizeof(T)), (StepShared<T, DP>::kWavesASimd)) void step_kernel(
    StepArgs a) {
  __shared__ __attribute__((aligned(16))) StepShared<T, DP> sh;
  step_body<T, DP, W>(a, int(blockIdx.x), sh);
}

// With the rows against those that all slots share in workgroups of the same launch, before the
// slots' own (neither fills the device: 64 answers on one document 39 us, in two launches 53 us).
template <typename T, int DP>
__global__ __launch_bounds__(kThreads, (StepShared<T, DP>::kWavesASimd)) void step_joint_kernel(StepArgs a) {
  using F = FwdShared<T, DP, 1>;
  using S = StepShared<T, DP>;
  __shared__ __attribute__((aligned(16))) char mem[sizeof(F) > sizeof(S) ? sizeof(F) : sizeof(S)];
  const int block = int(blockIdx.x);
  if (block < a.joint_blocks) {
    if (block < a.joint_items) fwd_body<T, DP, 1, false>(a.joint, block, *reinterpret_cast<F*>(mem));
  } else {
    step_body<T, DP, Op<T>::VE>(a, block - a.joint_blocks, *reinterpret_cast<S*>(mem));
  }
}

// ----------------------------------------------------------------- rows' join
//
// A workgroup takes 32 columns of one tile of rows, a thread 4 of one row: the parts
// against the row's own context, then those against the shared rows. Tiles of few rows
// (a token's heads) leave threads over, which take parts in turn and are joined in a
// fixed order. Bound: the parts' bytes; parts without a key are left out (their rows
// need not have been written).
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void rows_join_kernel(RowsJoinArgs a) {
  struct Sum {
    float m, l, e, v[4];
  };
  __shared__ Sum sums_of[kThreads];
  const Join j = ldc(a.own.joins + blockIdx.x);
  const Tile tl = ldc(a.own.qtiles + j.tile);
  const int lanes = tl.n <= 4 ? 4 : tl.n <= 8 ? 8 : tl.n <= 16 ? 16 : 32, turns = 32 / lanes;
  const int tid = int(threadIdx.x), n = tid / 8 % lanes, turn = tid / 8 / lanes;
  const int d = int(blockIdx.y) * 32 + tid % 8 * 4;
  const int row = tl.row0 + min(n, tl.n - 1), token = row / a.own.G, head = j.hk * a.own.G + row % a.own.G;
  int parts[2] = {j.parts, a.parts};
  int64_t own = int64_t(j.slot) * j.stride + j.within;
  int own_rows = 32;
  if (a.cut.lengths) {
    const StepTurns all = step_sum(a.cut);
    const int slot = j.tile / a.cut.tiles_a_slot, turns = step_turns(a.cut, ldc(a.cut.lengths + slot));
    const int share = step_share(a.cut, all.total);
    const int at = step_before(a.cut, all, slot) + j.tile % a.cut.tiles_a_slot * turns;
    const int i0 = at / share, i1 = (at + turns - 1) / share;  // workgroups
    if (turns > 0 && i0 == i1 && a.parts == 0) return;  // (final already)
    parts[0] = turns > 0 ? i1 - i0 + 1 : 0;
    if (turns == 0) parts[1] = 0;
    own_rows = min(a.own.G, 32);
    own = step_part(a.cut, j.hk, i0, j.tile);
  }
  const int64_t first[2] = {own * own_rows + row - tl.row0,
                            (int64_t(j.hk * a.units + row / 32 / max(a.per, 1)) * a.parts * a.per +
                             row / 32 % max(a.per, 1)) * 32 + row % 32};
  const int64_t step[2] = {int64_t(j.stride) * own_rows, int64_t(a.per) * 32};
  const float* const from[2] = {a.own.part, a.part};
  const float4* const sums[2] = {a.own.part_ml, a.part_ml};
  Sum s = {-INFINITY, 0.0f, 0.0f, {0, 0, 0, 0}};
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll 4
    for (int k = turn; k < parts[side]; k += turns) s.m = fmaxf(s.m, sums[side][first[side] + k * step[side]].x);
  float ref = s.m == -INFINITY ? 0.0f : s.m;
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll 4
    for (int k = turn; k < parts[side]; k += turns) {
      const int64_t r = first[side] + k * step[side];
      const float4 ml = sums[side][r];
      const f32x4 o = *reinterpret_cast<const f32x4*>(from[side] + r * DP + d);
      const bool some = ml.y != 0.0f;  // (NaN: some)
      const float w = exp2_fast(ml.x - ref);
      s.l += some ? ml.y * w : 0.0f;
      s.e += some ? ml.z * w : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) s.v[i] += some ? w * o[i] : 0.0f;
    }
  if (turns > 1) {
    sums_of[tid] = s;
    __syncthreads();
    if (turn > 0) return;
    // (turn 0's own top, not ref: that is 0 where its parts hold no key, and 2^(0 - all) times its
    // sums of 0 would be NaN for references below -128)
    const float own_top = s.m;
    for (int k = 1; k < turns; ++k) s.m = fmaxf(s.m, sums_of[tid + 8 * lanes * k].m);
    const float all = s.m == -INFINITY ? 0.0f : s.m;
    float w = exp2_fast(own_top - all);
    ref = all;
    s.l *= w;
    s.e *= w;
    for (int i = 0; i < 4; ++i) s.v[i] *= w;
    for (int k = 1; k < turns; ++k) {
      const Sum& o = sums_of[tid + 8 * lanes * k];
      w = exp2_fast(o.m - all);
      s.l += o.l * w;
      s.e += o.e * w;
      for (int i = 0; i < 4; ++i) s.v[i] += o.v[i] * w;
    }
  }
  if (n >= tl.n) return;
  const float inv = s.l > 0.0f || s.l != s.l ? 1.0f / s.l : 0.0f;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = s.v[i] * inv;
  scatter4(static_cast<T*>(a.own.out) + int64_t(token) * a.own.ldo, a.own.table, d, true, head, a.own.out_quad, v);
  if (a.own.lse && d == 0)
    a.own.lse[int64_t(token) * a.own.heads + head] =
        s.l > 0.0f || s.l != s.l ? (ref + __log2f(s.e)) * 0.69314718055994531f : -INFINITY;
}

// --------------------------------------------------------------------- delta
//
// rowsum(grad_out out) of queries that see few keys, from its other form sum_j P_ij dP_ij:
// the stored out is rounded to bf16, and where few keys share a row that rounding is as
// large as the score gradients it is taken from (a causal training batch's grad_q and grad_k 0.0025
// off, with this 0.0024). A workgroup takes a tile of query rows, a wave one of its key tiles.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads, few_waves(DP, sizeof(T))) void delta_kernel(BwdArgs a, const int4* tiles,
                                                                                   float* rows) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  __shared__ float sums[4][64];
  const int4 it = ldc(tiles + blockIdx.x);  // tile, first and end of its key tiles
  const int hk = int(blockIdx.y), lane = lane_id(), n = lane % 32, h = lane / 32, wave = wave_id();
  const Tile tl = ldc(a.qtiles + it.x);
  const Reach re = ldc(a.reach + it.x);
  const int64_t qat = int64_t(it.x) * a.groups + hk;
  float sum = 0.0f;
  if (it.y + wave < it.z) {
    const int t = it.y + wave, tile = key_tile<true>(a, re.skip, t);
    const int64_t at = (int64_t(tile) * a.groups + hk) * D::TILE;
    const float lse2 = a.rows[qat * 64 + n];
    f32x16 s = zero16(), dp = zero16();
#pragma unroll
    for (int u = 0; u < D::KSTEPS; ++u) {
      s = Op<T>::mma(as_frag<Frag>(unit16(a.kforms<T>(kKRows) + at, u, lane)),
                     as_frag<Frag>(unit16(a.qforms<T>(kQRows) + qat * D::TILE, u, lane)), s);
      dp = Op<T>::mma(as_frag<Frag>(unit16(a.kforms<T>(kVRows) + at, u, lane)),
                      as_frag<Frag>(unit16(a.qforms<T>(kGRows) + qat * D::TILE, u, lane)), dp);
    }
    const int hidden = a.causal ? hidden_from(a, re, tl.row0 + min(n, tl.n - 1)) : INT_MAX;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 8 * (i / 4) + 4 * h + i % 4;
      const bool seen = (t < a.shared || 32 * tile + r < hidden) && a.bias[int64_t(tile) * 32 + r] >= 0.0f;
      const float p = exp2_fast(s[i] * a.scale2 - lse2);
      sum += seen ? p * dp[i] : 0.0f;
    }
    sum = half_sum(sum);
  }
  sums[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && h == 0) rows[qat * 64 + 32 + n] = sums[0][n] + sums[1][n] + (sums[2][n] + sums[3][n]);
}

// -------------------------------------------------------------------- launch

template <typename T, int DP>
struct SeqKernels {
  static void step_sums(const StepCut& c, hipStream_t s) {
    hipLaunchKernelGGL(step_sums_kernel, dim3(1), dim3(kSumThreads), 0, s, c);
  }
  static void pack(const PackArgs& a, hipStream_t s) {
    const bool grads = a.rows_out != nullptr, vec = a.t[0].vec && a.t[1].vec && (!grads || a.out_vec);
    const auto k = vec ? (grads ? pack_kernel<T, DP, true, true, true> : pack_kernel<T, DP, true, false, true>)
                       : (grads ? pack_kernel<T, DP, false, true, true> : pack_kernel<T, DP, false, false, true>);
    hipLaunchKernelGGL(k, dim3(unsigned((a.ntiles + 7) / 8 * 8 * a.groups)), dim3(kThreads), 0, s, a);
  }
  static void delta(const BwdArgs& a, const int4* tiles, int count, float* rows, hipStream_t s) {
    hipLaunchKernelGGL((delta_kernel<T, DP>), dim3(unsigned(count), unsigned(a.groups)), dim3(kThreads), 0, s, a, tiles, rows);
  }
  static void fwd(const FwdArgs& a, int items, int tiles, hipStream_t s) {
    if (tiles == 1) hipLaunchKernelGGL((fwd_few_kernel<T, DP, true>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
    if (tiles == 4) hipLaunchKernelGGL((fwd_kernel<T, DP, 1, true>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
    if constexpr (wide_forward(DP, sizeof(T)))
      if (tiles == 8) hipLaunchKernelGGL((fwd_kernel<T, DP, 2, true>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
  }
  static void bwd(const BwdArgs& a, int items, hipStream_t s) {
    hipLaunchKernelGGL((bwd_kernel<T, DP, true>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
    if (!a.causal) return;
    // four tiles an item, four waves a workgroup: one tile a wave, and more from 768 workgroups on
    const int shift = items <= 768 ? 0 : items <= 2 * 768 ? 1 : items <= 4 * 768 ? 2 : 3, per = 1 << shift;
    hipLaunchKernelGGL((redo_kernel<T, DP>), dim3(unsigned((items + per - 1) / per)), dim3(kThreads), 0, s, a, items, shift);
  }
  static void step(const StepArgs& a, hipStream_t s) {
    const unsigned groups = a.whole ? unsigned(a.cut.slots) * unsigned(a.cut.tiles_a_slot) : unsigned(a.cut.shares);
    const dim3 grid((groups + 7) / 8 * 8 * unsigned(a.bundles) + unsigned(a.joint_blocks));
    const dim3 threads(64 * step_waves(DP, sizeof(T)));
    if constexpr (step_with_joint(DP, sizeof(T)))
      if (a.joint_blocks) {
        hipLaunchKernelGGL((step_joint_kernel<T, DP>), grid, threads, 0, s, a);
        return;
      }
    if (a.width == Op<T>::VE)
      hipLaunchKernelGGL((step_kernel<T, DP, Op<T>::VE>), grid, threads, 0, s, a);
    else if (sizeof(T) == 2 && a.width == 4)
      hipLaunchKernelGGL((step_kernel<T, DP, 4>), grid, threads, 0, s, a);
    else
      hipLaunchKernelGGL((step_kernel<T, DP, 1>), grid, threads, 0, s, a);
  }
  static void rows_join(const RowsJoinArgs& a, int joins, hipStream_t s) {
    hipLaunchKernelGGL((rows_join_kernel<T, DP>), dim3(unsigned(joins), DP / 32), dim3(kThreads), 0, s, a);
  }
  static SeqTable table() {
    if constexpr (sizeof(T) == 2) return {pack, fwd, bwd, step_sums, step, rows_join, delta};
    else return {pack, fwd, bwd, step_sums, step, rows_join, nullptr};
  }
};

}  // namespace attn
}  // namespace cgtp
