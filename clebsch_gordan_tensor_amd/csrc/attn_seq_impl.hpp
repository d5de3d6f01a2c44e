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

// Quads: 4 keys x VE channels from rows in registers to VE columns of 4 keys.
template <typename T>
struct Quad;
template <>
struct Quad<bf16> {
  static constexpr int kStride = 80;  // bytes a column: 32 keys and 16 against bank conflicts
  // Byte of quad q in column d: column fragment f, half h hold quads 4 f + h and
  // 4 f + 2 + h next to each other, as 16 bytes whose place turns with d / 16: the columns of
  // 16 bytes of a row start at two banks only.
  static __device__ __forceinline__ int at(int d, int q) {
    return d * kStride + ((q / 4 * 2 + q % 2) ^ (d / 16 & 3)) * 16 + q / 2 % 2 * 8;
  }
  static __device__ __forceinline__ int frag(int d, int f, int h) {
    return d * kStride + ((2 * f + h) ^ (d / 16 & 3)) * 16;
  }
  static __device__ __forceinline__ void turn(const u32x4 (&r)[4], char* column) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t a = r[0][c], b = r[1][c], d = r[2][c], e = r[3][c];
      uint2 lo, hi;
      lo.x = __builtin_amdgcn_perm(b, a, 0x05040100);
      lo.y = __builtin_amdgcn_perm(e, d, 0x05040100);
      hi.x = __builtin_amdgcn_perm(b, a, 0x07060302);
      hi.y = __builtin_amdgcn_perm(e, d, 0x07060302);
      *reinterpret_cast<uint2*>(column + 2 * c * kStride) = lo;
      *reinterpret_cast<uint2*>(column + (2 * c + 1) * kStride) = hi;
    }
  }
};
template <>
struct Quad<float> {
  static constexpr int kStride = 144;
  static __device__ __forceinline__ int at(int d, int q) { return d * kStride + (q ^ (d / 16 & 7)) * 16; }
  static __device__ __forceinline__ int frag(int d, int f, int h) { return at(d, 2 * f + h); }
  static __device__ __forceinline__ void turn(const u32x4 (&r)[4], char* column) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<u32x4*>(column + c * kStride) = u32x4{r[0][c], r[1][c], r[2][c], r[3][c]};
  }
};

// Elements d0 .. d0 + VE - 1 of a context row's head; those outside the head are 0.
template <typename T>
__device__ __forceinline__ u32x4 row_piece(const T* row, const int4* table, int d0, int head, int size) {
  constexpr int VE = Op<T>::VE;
  u32x4 v;
  T t[VE];
#pragma unroll
  for (int j = 0; j < VE; ++j) t[j] = row[elem(table[d0 + j], false, head)];
  __builtin_memcpy(&v, t, 16);
  return inside_head<T, false>(v, d0, size);
}

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
  const int run = slot / s.each;
  int n = __builtin_amdgcn_readlane(s.upto - s.mine, run);
  for (int i = run * s.each; i < slot; ++i) n += step_turns(c, ldc(c.lengths + i)) * c.tiles_a_slot;
  return n;
}
// The slot that turn `at` (below the total) belongs to, and its first turn.
__device__ __forceinline__ int2 step_find(const StepCut& c, const StepTurns& s, int at) {
  const int run = __builtin_ctzll(__ballot(s.upto > at));
  int slot = run * s.each, n = __builtin_amdgcn_readlane(s.upto - s.mine, run);
  while (true) {
    const int turns = step_turns(c, ldc(c.lengths + slot)) * c.tiles_a_slot;
    if (n + turns > at) return make_int2(slot, n);
    n += turns;
    ++slot;
  }
}

// The first of the parts (one for each wave of the head) of workgroup `index` and tile of rows qt.
__device__ __forceinline__ int step_part(const StepCut& c, int hk, int index, int qt) {
  return (hk * (c.shares + c.slots * c.tiles_a_slot) + index + qt) * c.waves_a_head;
}

// What a workgroup does next: turns a .. b - 1 of tile of rows qt.
struct StepWork {
  int hk;   // this wave's context head
  bool on;  // (the last workgroup of a row may have fewer heads than waves)
  int index, bundle, at, end;
  int slot, before;  // the slot of turn `at` and the turns before it
  int qt, len, t0, t1;  // key tiles t0 .. t1 - 1
  bool last;            // the slot's last places are among them
  Item it;
};
// False: the workgroup has nothing to do.
__device__ __forceinline__ bool step_begin(const StepArgs& a, int wave, StepWork& w) {
  const int turn = int(blockIdx.x) / 8;
  w.bundle = turn % a.bundles;
  w.index = turn / a.bundles * 8 + int(blockIdx.x) % 8;
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
    w.last = turns > 0;
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
  w.last = last == turns;
  const bool alone = first == 0 && last == turns && wph == 1 && !a.joined;
  w.it = {w.qt, 1, w.t0, w.t1, w.hk, alone ? -1 : step_part(a.cut, w.hk, w.index, w.qt) + wave % wph, 1, 0};
  return true;
}

template <typename T>
struct StepRows {
  const T *cache, *fresh;
  int64_t dim;
  int len;
  // the new row at the end, also for places behind it, which are hidden
  __device__ __forceinline__ const T* at(int key) const { return key >= len ? fresh : cache + int64_t(key) * dim; }
};
template <typename T>
__device__ __forceinline__ StepRows<T> step_rows(const StepArgs& a, const StepWork& w, const void* cache,
                                                 const void* fresh, int64_t ld) {
  return {static_cast<const T*>(cache) + int64_t(w.slot) * a.cut.capacity * a.dim,
          static_cast<const T*>(fresh) + w.slot * ld, a.dim, w.len};
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
      const u32x4 x = *reinterpret_cast<const u32x4*>(columns + Quad<T>::frag(32 * d + lane % 32, f, lane / 32));
      st.o[d] = Op<T>::mma(as_frag<typename Op<T>::Frag>(x), w[f], st.o[d]);
    }
}

// Whether the registers hold the next turn's rows.
constexpr bool step_ahead(int dp, size_t size) { return dp * int(size) <= 512 && dp <= 192; }

// Bytes of shared memory of a step's waves: a row of keys, a wave's rows, its columns of values
// (with paddings against bank conflicts).
constexpr int step_row(int dp, size_t size) { return dp * int(size) + 16; }
constexpr int step_rows_bytes(int dp, size_t size) { return 32 * step_row(dp, size) + 64; }
template <typename T>
constexpr int step_columns_bytes(int dp) { return dp * Quad<T>::kStride + 64; }
template <typename T>
constexpr int step_waves_a_simd(int dp) {
  return step_waves(dp, sizeof(T)) * (step_rows_bytes(dp, sizeof(T)) + step_columns_bytes<T>(dp)) <= 80 * 1024
             ? few_waves(dp, sizeof(T)) : 1;
}

// Rows whose heads are whole aligned 16-byte pieces. The workgroup reads the rows of its
// heads in their order in memory, quads of 4 keys x 16 bytes a lane, a turn ahead in
// registers (reading every head's pieces straight as operands took twice as long: each load
// then touches 64 cache lines), and lays them out in shared memory: keys by rows, values
// by columns, each wave's tile in a place of its own.
template <typename T, int DP>
__global__ __launch_bounds__(64 * step_waves(DP, sizeof(T)), step_waves_a_simd<T>(DP)) void step_kernel(StepArgs a) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  using Q = Quad<T>;
  constexpr int VE = D::VE, WAVES = step_waves(DP, sizeof(T)), PER = (DP / VE + 7) / 8;
  constexpr int ROW = step_row(DP, sizeof(T)), ROWS = step_rows_bytes(DP, sizeof(T)), COLUMNS = step_columns_bytes<T>(DP);
  __shared__ __attribute__((aligned(16))) char key_rows[WAVES][ROWS], columns[WAVES][COLUMNS];
  StepWork w;
  const int tid = int(threadIdx.x), wave = wave_id(), lane = lane_id(), n = lane % 32, h = lane / 32;
  if (!step_begin(a, wave, w)) return;
  const int wph = a.cut.waves_a_head;
  const int hk0 = w.hk - wave / wph, heads = min(a.heads_a_group, a.f.groups - hk0);
  // quads of this thread: one piece of four keys each (threads without one, and those of
  // heads that the last workgroup of a row does not have, repeat another's)
  const int row_bytes = int(a.dim * int64_t(sizeof(T)));
  int key[PER], row_at[PER], column_at[PER];
  uint32_t off[PER];  // bytes from the row's start
#pragma unroll
  for (int g = 0; g < PER; ++g) {
    const int i = (tid + 64 * WAVES * g) % (8 * wph * a.pieces), quad = i / a.pieces;
    StepPiece p = a.piece[i % a.pieces];
    if (p.j >= heads) p = a.piece[0];
    key[g] = 4 * quad;
    off[g] = uint32_t(p.off + hk0 * p.cw) * uint32_t(sizeof(T));
    const int place = p.j * wph + quad / 8;
    row_at[g] = place * ROWS + quad % 8 * 4 * ROW + p.d * int(sizeof(T));
    column_at[g] = place * COLUMNS + Q::at(p.d, quad % 8);
  }
  // Quads first .. first + count - 1 of the turn from tile t on. Places behind the
  // sequence's end are read as well (they are hidden), but none behind the caches' end.
  const auto load = [&](const void* cache, int t, auto first, auto count, u32x4 (&x)[decltype(count)::value][4]) {
    const int64_t row = int64_t(w.slot) * a.cut.capacity + int64_t(t) * 32;
    const char* const base = static_cast<const char*>(cache) + row * row_bytes;
    const int rows = int(min(int64_t(a.cut.slots) * a.cut.capacity - row, int64_t(32 * WAVES)));
#pragma unroll
    for (int i = 0; i < decltype(count)::value; ++i) {
      const int g = decltype(first)::value + i;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[i][r] = *reinterpret_cast<const u32x4*>(
            base + (off[g] + (key[g] + r < rows ? uint32_t(key[g] + r) * uint32_t(row_bytes) : 0u)));
    }
  };
  const auto put_keys = [&](auto first, auto count, const u32x4 (&x)[decltype(count)::value][4]) {
#pragma unroll
    for (int i = 0; i < decltype(count)::value; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<u32x4*>(&key_rows[0][0] + row_at[decltype(first)::value + i] + r * ROW) = x[i][r];
  };
  const auto put_values = [&](int t, auto first, auto count, u32x4 (&x)[decltype(count)::value][4]) {
    // weight 0 times what a place from the end on holds would be NaN for infinities
    if (32 * (t + wph) > w.len)
#pragma unroll
      for (int i = 0; i < decltype(count)::value; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          x[i][r] = 32 * t + key[decltype(first)::value + i] + r >= w.len ? u32x4{0, 0, 0, 0} : x[i][r];
#pragma unroll
    for (int i = 0; i < decltype(count)::value; ++i)
      Q::turn(x[i], &columns[0][0] + column_at[decltype(first)::value + i]);
  };
  using none = std::integral_constant<int, 0>;
  using every = std::integral_constant<int, PER>;
  // the widest heads leave no registers for the next turn's rows
  constexpr bool kAhead = step_ahead(DP, sizeof(T));
  constexpr int HELD = kAhead ? PER : 1;
  // both tensors' rows of a turn, half of the quads at a time
  const auto pass = [&](int t, auto first, auto count) {
    u32x4 x[decltype(count)::value][4];
    load(a.k_cache, t, first, count, x);
    put_keys(first, count, x);
    __builtin_amdgcn_sched_barrier(0);
    load(a.v_cache, t, first, count, x);
    put_values(t, first, count, x);
    __builtin_amdgcn_sched_barrier(0);
  };
  // (keys' places beyond the head meet zeros of the queries, and must not be NaN)
  if (a.size < DP)
    for (int i = lane; i < 32 * (DP - a.size); i += 64)
      *reinterpret_cast<T*>(&key_rows[wave][i % 32 * ROW + (a.size + i / 32) * int(sizeof(T))]) = T{};
  const bool exact = sizeof(T) == 2 && a.f.lse != nullptr;
  while (step_next(a, wave, w)) {
    u32x4 k[HELD][4], v[HELD][4];
    if constexpr (kAhead)
      if (w.t0 < w.t1) {
        load(a.k_cache, w.t0, none{}, every{}, k);
        load(a.v_cache, w.t0, none{}, every{}, v);
      }
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
        put_keys(none{}, every{}, k);
        load(a.k_cache, next, none{}, every{}, k);
        put_values(t, none{}, every{}, v);
        load(a.v_cache, next, none{}, every{}, v);
      } else {
        using half = std::integral_constant<int, PER / 2>;
        pass(t, none{}, half{});
        pass(t, half{}, std::integral_constant<int, PER - PER / 2>{});
      }
      turn_lds();
      if (w.on && mine < w.t1) {
        if (mine == w.len / 32) {
          const int r = w.len % 32;
          take_new<T>(a, w, [&](int d, T x, T y) {
            *reinterpret_cast<T*>(&key_rows[wave][r * ROW + d * int(sizeof(T))]) = x;
            *reinterpret_cast<T*>(&columns[wave][Q::at(d, r / 4) + r % 4 * int(sizeof(T))]) = y;
          });
          wave_fence();
        }
        f32x16 sc = zero16();
#pragma unroll
        for (int u = 0; u < D::KSTEPS; ++u) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(&key_rows[wave][n * ROW + (2 * u + h) * 16]);
          sc = Op<T>::mma(as_frag<Frag>(x), q[u], sc);
        }
        Frag p[D::FR];
        step_weigh<T, DP>(a, mine, w.len, st, sc, e, exact, p);
        step_values<T, DP>(columns[wave], lane, st, p);
      }
      turn_lds();
    }
    if (w.on) finish<T, DP>(a.f, w.it, tl, 0, st, e, min(a.f.G, 32));
  }
}

// Rows of any alignment, read element by element: keys straight as operands, values
// turned in a wave's own place.
template <typename T, int DP>
__global__ __launch_bounds__(64 * step_waves(DP, sizeof(T)), few_waves(DP, sizeof(T))) void step_elements_kernel(
    StepArgs a) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  using Q = Quad<T>;
  constexpr int VE = D::VE, PIECES = DP / VE, PER = (PIECES + 7) / 8;
  __shared__ __attribute__((aligned(16))) char columns[step_waves(DP, sizeof(T))][DP * Q::kStride];
  StepWork w;
  const int wave = wave_id(), lane = lane_id(), n = lane % 32;
  if (!step_begin(a, wave, w) || !w.on) return;
  char* const mine = columns[wave];
  const bool exact = sizeof(T) == 2 && a.f.lse != nullptr;
  while (step_next(a, wave, w)) {
    const auto kr = step_rows<T>(a, w, a.k_cache, a.k_new, a.ldk), vr = step_rows<T>(a, w, a.v_cache, a.v_new, a.ldv);
    const Tile tl = ldc(a.f.qtiles + w.qt);
    Frag q[D::KSTEPS];
    load_queries<T, DP>(a.f, tl, w.hk, lane, q);
    Running<D::DT> st;
    float e = 0.0f;
#pragma unroll
    for (int d = 0; d < D::DT; ++d) st.o[d] = zero16();
    for (int t = w.t0 + wave % a.cut.waves_a_head; t < w.t1; t += a.cut.waves_a_head) {
      f32x16 sc = zero16();
#pragma unroll
      for (int u = 0; u < D::KSTEPS; ++u) {
        const u32x4 x = row_piece<T>(kr.at(32 * t + n), a.f.table, VE * (2 * u + lane / 32), w.hk, a.size);
        sc = Op<T>::mma(as_frag<Frag>(x), q[u], sc);
        if (u % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
      Frag p[D::FR];
      step_weigh<T, DP>(a, t, w.len, st, sc, e, exact, p);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = lane + 64 * i, piece = c / 8, quad = c % 8;
        if (PIECES % 8 != 0 && piece >= PIECES) break;
        u32x4 x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = 32 * t + 4 * quad + r;
          x[r] = row_piece<T>(vr.at(key), a.f.table, VE * piece, w.hk, a.size);
          if (key > w.len) x[r] = u32x4{0, 0, 0, 0};
        }
        Q::turn(x, mine + Q::at(VE * piece, quad));
        __builtin_amdgcn_sched_barrier(0);
      }
      wave_fence();
      step_values<T, DP>(mine, lane, st, p);
      wave_fence();
    }
    if (w.last && wave % a.cut.waves_a_head == 0) take_new<T>(a, w, [](int, T, T) {});
    finish<T, DP>(a.f, w.it, tl, 0, st, e, min(a.f.G, 32));
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
    if (turns > 0 && i0 == i1 && a.cut.waves_a_head == 1 && a.parts == 0) return;  // (final already)
    parts[0] = turns > 0 ? (i1 - i0 + 1) * a.cut.waves_a_head : 0;
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
    for (int k = 1; k < turns; ++k) s.m = fmaxf(s.m, sums_of[tid + 8 * lanes * k].m);
    const float all = s.m == -INFINITY ? 0.0f : s.m;
    float w = exp2_fast(ref - all);
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

// -------------------------------------------------------------------- launch

template <typename T, int DP>
struct SeqKernels {
  static void fwd(const FwdArgs& a, int items, int tiles, hipStream_t s) {
    if (tiles == 1) hipLaunchKernelGGL((fwd_few_kernel<T, DP, true>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
    if (tiles == 4) hipLaunchKernelGGL((fwd_kernel<T, DP, 1, true>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
    if constexpr (wide_forward(DP, sizeof(T)))
      if (tiles == 8) hipLaunchKernelGGL((fwd_kernel<T, DP, 2, true>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
  }
  static void bwd(const BwdArgs& a, int items, hipStream_t s) {
    hipLaunchKernelGGL((bwd_kernel<T, DP, true>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
  }
  static void step(const StepArgs& a, hipStream_t s) {
    const unsigned groups = a.whole ? unsigned(a.cut.slots) * unsigned(a.cut.tiles_a_slot) : unsigned(a.cut.shares);
    const dim3 grid((groups + 7) / 8 * 8 * unsigned(a.bundles));
    const dim3 threads(64 * step_waves(DP, sizeof(T)));
    if (a.vec) hipLaunchKernelGGL((step_kernel<T, DP>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((step_elements_kernel<T, DP>), grid, threads, 0, s, a);
  }
  static void rows_join(const RowsJoinArgs& a, int joins, hipStream_t s) {
    hipLaunchKernelGGL((rows_join_kernel<T, DP>), dim3(unsigned(joins), DP / 32), dim3(kThreads), 0, s, a);
  }
  static SeqTable table() { return {fwd, bwd, step, rows_join}; }
};

}  // namespace attn
}  // namespace cgtp
