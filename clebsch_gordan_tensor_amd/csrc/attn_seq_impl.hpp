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
// into the cache by the wave whose part of the places it ends. A wave takes one tile of
// query rows (the heads that share a context head) and one part of the places, 32 keys a
// turn: S^T = K Q^T with the keys' rows as operands straight from memory (16 bytes a
// lane), O^T += V^T P^T with the values turned by way of shared memory (quads of keys,
// a wave's own place, so no barrier). The rows stay as the caller has them: no packing,
// and a cache can be read, copied or cut with ordinary tensor operations.
//
// Bound: the cached rows' bytes. A head's channels are short runs of a row (16 bytes for
// 32 channels over 4 heads in bf16), so the waves of a workgroup take neighbouring heads of the
// same places, whose runs lie in the same cache lines, and the other heads' workgroups follow on
// the same die (workgroup index modulo 8).

// Quads: 4 keys x VE channels from rows in registers to VE columns of 4 keys.
template <typename T>
struct Quad;
template <>
struct Quad<bf16> {
  static constexpr int kStride = 80;  // bytes a column: 32 keys and 16 against bank conflicts
  static constexpr int kBytes = 8;
  // place of quad q in a column: column fragment f, half h hold quads 4 f + h and 4 f + 2 + h
  static __device__ __forceinline__ int slot(int q) { return q / 4 * 4 + q % 2 * 2 + q / 2 % 2; }
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
  static constexpr int kBytes = 16;
  static __device__ __forceinline__ int slot(int q) { return q; }
  static __device__ __forceinline__ void turn(const u32x4 (&r)[4], char* column) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<u32x4*>(column + c * kStride) = u32x4{r[0][c], r[1][c], r[2][c], r[3][c]};
  }
};

// Elements d0 .. d0 + VE - 1 of a context row's head; those outside the head are 0.
template <typename T, bool VEC>
__device__ __forceinline__ u32x4 row_piece(const T* row, const int4* table, int d0, int head, int size) {
  constexpr int VE = Op<T>::VE;
  u32x4 v;
  if constexpr (VEC) {
    v = *reinterpret_cast<const u32x4*>(row + elem(table[d0], false, head));
  } else {
    T t[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) t[j] = row[elem(table[d0 + j], false, head)];
    __builtin_memcpy(&v, t, 16);
  }
  return inside_head<T, VEC>(v, d0, size);
}

// Orders a wave's own writes and reads of shared memory.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(kThreads, few_waves(DP, sizeof(T))) void step_kernel(StepArgs a) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  using Q = Quad<T>;
  constexpr int VE = D::VE, PIECES = DP / VE, PER = (PIECES + 7) / 8;  // quads of pieces a lane
  __shared__ __attribute__((aligned(16))) char columns[4][DP * Q::kStride];
  const int turn = int(blockIdx.x) / 8, bundle = turn % a.bundles;
  int at = turn / a.bundles * 8 + int(blockIdx.x) % 8;
  if (at >= a.slots * a.tiles_a_slot * a.splits) return;
  const int split = at % a.splits;
  at /= a.splits;
  const int qt = at, slot = at / a.tiles_a_slot, wave = wave_id(), lane = lane_id(), n = lane % 32, h = lane / 32;
  const int hk = bundle * a.heads_a_group + wave / a.waves_a_head;
  if (wave / a.waves_a_head >= a.heads_a_group || hk >= a.f.groups) return;
  const int parts = a.splits * a.waves_a_head, p = split * a.waves_a_head + wave % a.waves_a_head;
  const int len = ldc(a.lengths + slot);
  const bool used = len >= 0 && len < a.capacity;
  const int nt = used ? len / 32 + 1 : 0, per = max(a.min_tiles, (nt + parts - 1) / parts);
  const int t0 = min(p * per, nt), t1 = min(t0 + per, nt);
  const Tile tl = ldc(a.f.qtiles + qt);
  const Item it = {qt, 1, t0, t1, hk, a.whole ? -1 : (qt * a.f.groups + hk) * parts + p, 1, 0};
  const T* const k_rows = static_cast<const T*>(a.k_cache) + int64_t(slot) * a.capacity * a.dim;
  const T* const v_rows = static_cast<const T*>(a.v_cache) + int64_t(slot) * a.capacity * a.dim;
  const T* const k_new = static_cast<const T*>(a.k_new) + slot * a.ldk;
  const T* const v_new = static_cast<const T*>(a.v_new) + slot * a.ldv;
  const auto row = [&](const T* rows, const T* fresh, int key) {
    return key >= len ? fresh : rows + int64_t(key) * a.dim;  // (places behind the new one are hidden)
  };
  char* const mine = columns[wave];

  const auto load_k = [&](int t, int u) {
    return row_piece<T, VEC>(row(k_rows, k_new, 32 * t + n), a.f.table, 2 * VE * u + VE * h, hk, a.size);
  };
  // quad i of this lane: piece and its four keys
  const auto load_v = [&](int t, int i, u32x4 (&v)[4]) {
    const int c = lane + 64 * i, piece = min(c / 8, PIECES - 1), q = c % 8;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      v[r] = row_piece<T, VEC>(row(v_rows, v_new, 32 * t + 4 * q + r), a.f.table, VE * piece, hk, a.size);
  };
  const auto turn_v = [&](int t, int i, u32x4 (&v)[4]) {
    const int c = lane + 64 * i, piece = c / 8, q = c % 8;
    if (PIECES % 8 != 0 && piece >= PIECES) return;
    // weight 0 times what such a row holds would be NaN for infinities
    if (32 * t + 31 > len)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = 32 * t + 4 * q + r > len ? u32x4{0, 0, 0, 0} : v[r];
    Q::turn(v, mine + VE * piece * Q::kStride + Q::slot(q) * Q::kBytes);
  };
  // the widest heads leave no registers for whole tiles: read as they are used
  constexpr bool kStream = DP * int(sizeof(T)) > 512 || !VEC;
  u32x4 k[kStream ? 1 : D::KSTEPS], v[kStream ? 1 : PER][4];
  const auto fetch_k = [&](int t) {
    if constexpr (!kStream)
#pragma unroll
      for (int u = 0; u < D::KSTEPS; ++u) k[u] = load_k(t, u);
  };
  const auto fetch_v = [&](int t) {
    if constexpr (!kStream)
#pragma unroll
      for (int i = 0; i < PER; ++i) load_v(t, i, v[i]);
  };
  if (t0 < t1) {
    fetch_k(t0);
    fetch_v(t0);
  }
  Frag q[D::KSTEPS];
  load_queries<T, DP>(a.f, tl, hk, lane, q);
  Running<D::DT> st;
  float e = 0.0f;
  const bool exact = sizeof(T) == 2 && a.f.lse != nullptr;
#pragma unroll
  for (int d = 0; d < D::DT; ++d) st.o[d] = zero16();
  for (int t = t0; t < t1; ++t) {
    const int next = min(t + 1, t1 - 1);
    f32x16 sc = zero16();
#pragma unroll
    for (int u = 0; u < D::KSTEPS; ++u) {
      if constexpr (kStream) {
        sc = Op<T>::mma(as_frag<Frag>(load_k(t, u)), q[u], sc);
        if (u % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      } else {
        sc = Op<T>::mma(as_frag<Frag>(k[u]), q[u], sc);
      }
    }
    fetch_k(next);
    if (32 * t + 31 > len) hide_later(sc, t, len + 1, h);
    raise_reference(st, top_score(sc, a.f.scale2), e, exact);
    Frag w[D::FR];
    weigh<T, true>(st, sc, a.f.scale2, 0.0f, e, exact, w);
    if constexpr (kStream) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        u32x4 x[4];
        load_v(t, i, x);
        turn_v(t, i, x);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) turn_v(t, i, v[i]);
    }
    wave_fence();
    fetch_v(next);
#pragma unroll
    for (int d = 0; d < D::DT; ++d)
#pragma unroll
      for (int f = 0; f < D::FR; ++f) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(mine + (32 * d + n) * Q::kStride + (2 * f + h) * 16);
        st.o[d] = Op<T>::mma(as_frag<Frag>(x), w[f], st.o[d]);
      }
    wave_fence();
  }
  // the new rows' elements of this head, by the wave that holds the last place
  if (t0 < t1 && t1 == nt && qt % a.tiles_a_slot == 0) {
    T* const ko = static_cast<T*>(a.k_cache) + (int64_t(slot) * a.capacity + len) * a.dim;
    T* const vo = static_cast<T*>(a.v_cache) + (int64_t(slot) * a.capacity + len) * a.dim;
    for (int d = lane; d < a.size; d += 64) {
      const int64_t i = elem(a.f.table[d], false, hk);
      ko[i] = k_new[i];
      vo[i] = v_new[i];
    }
  }
  finish<T, DP>(a.f, it, tl, 0, st, e);
}

// ----------------------------------------------------------------- rows' join
//
// A workgroup takes 32 columns of one tile of rows, a thread 4 of one row: the parts
// against the row's own context, then those against the shared rows. Bound: the parts'
// bytes. Parts without a key are left out (their rows need not have been written).
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void rows_join_kernel(RowsJoinArgs a) {
  const Join j = ldc(a.own.joins + blockIdx.x);
  const Tile tl = ldc(a.own.qtiles + j.tile);
  const int n = int(threadIdx.x) / 8, d = int(blockIdx.y) * 32 + int(threadIdx.x) % 8 * 4;
  if (n >= tl.n) return;
  const int row = tl.row0 + n, token = row / a.own.G, head = j.hk * a.own.G + row % a.own.G;
  const int len = a.lengths ? a.lengths[token] : 0;
  const bool none = a.lengths && (len < 0 || len >= a.capacity);
  const int64_t first[2] = {(int64_t(j.slot) * j.stride + j.within) * 32 + n,
                            (int64_t(j.hk * a.units + row / 32 / max(a.per, 1)) * a.parts * a.per +
                             row / 32 % max(a.per, 1)) * 32 + row % 32};
  const int64_t step[2] = {int64_t(j.stride) * 32, int64_t(a.per) * 32};
  const int parts[2] = {none ? 0 : j.parts, none ? 0 : a.parts};
  const float* const from[2] = {a.own.part, a.part};
  const float4* const sums[2] = {a.own.part_ml, a.part_ml};
  float m = -INFINITY, l = 0.0f, e = 0.0f;
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll 4
    for (int k = 0; k < parts[side]; ++k) m = fmaxf(m, sums[side][first[side] + k * step[side]].x);
  const float ref = m == -INFINITY ? 0.0f : m;
  float v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll 4
    for (int k = 0; k < parts[side]; ++k) {
      const int64_t r = first[side] + k * step[side];
      const float4 ml = sums[side][r];
      const f32x4 o = *reinterpret_cast<const f32x4*>(from[side] + r * DP + d);
      const bool some = ml.y != 0.0f;  // (NaN: some)
      const float w = exp2_fast(ml.x - ref);
      l += some ? ml.y * w : 0.0f;
      e += some ? ml.z * w : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += some ? w * o[i] : 0.0f;
    }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] *= inv;
  scatter4(static_cast<T*>(a.own.out) + int64_t(token) * a.own.ldo, a.own.table, d, true, head, a.own.out_quad, v);
  if (a.own.lse && d == 0)
    a.own.lse[int64_t(token) * a.own.heads + head] =
        l > 0.0f || l != l ? (ref + __log2f(e)) * 0.69314718055994531f : -INFINITY;
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
    const unsigned groups = unsigned(a.slots) * unsigned(a.tiles_a_slot) * unsigned(a.splits);
    const dim3 grid((groups + 7) / 8 * 8 * unsigned(a.bundles));
    if (a.vec) hipLaunchKernelGGL((step_kernel<T, DP, true>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((step_kernel<T, DP, false>), grid, dim3(kThreads), 0, s, a);
  }
  static void rows_join(const RowsJoinArgs& a, int joins, hipStream_t s) {
    hipLaunchKernelGGL((rows_join_kernel<T, DP>), dim3(unsigned(joins), DP / 32), dim3(kThreads), 0, s, a);
  }
  static SeqTable table() { return {fwd, bwd, step, rows_join}; }
};

}  // namespace attn
}  // namespace cgtp
