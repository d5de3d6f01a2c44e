// Cross attention on irreps rows: kernels templated on storage type and padded
// head size (instantiated in inst/attn_*.hip, launched by attn_kernels.hip).
//
// For a query row (one query, one head) and the keys of its sample:
//   s_j = scale q.k_j,  p = softmax s,  o = sum_j p_j v_j
// A row of 32 queries x a tile of 32 keys is one matrix-core tile. The kernels
// compute S^T = K Q^T, so that a lane holds one query (column lane % 32) and 16
// of the tile's keys, reduces over keys mostly inside the lane, and feeds the
// same registers as the B operand of O^T += V^T P^T: no exchange between lanes
// and no shared memory for P.
//
// The keys come packed in "fragments", the order in which a wave reads a matrix
// operand: 1 KB units of 64 lanes x 16 bytes (VE = 8 bf16 or 4 fp32 values).
//   row fragment t of a 32 x DP tile:    lane l holds [l % 32][2 VE t + VE h + j]
//   column fragment (dt, f) of the tile: lane l holds, for column 32 dt + l % 32,
//       the rows 8 (r / 4) + 4 h + r % 4 with r = VE f + j
// (h = l / 32, j = 0 .. VE - 1; the row order of the second is the one in which
// the accumulator registers of S^T hold the keys). Packing gathers a head's
// channels out of the irreps blocks, pads heads to DP and tiles to 32 rows with
// zeros and writes zeros for masked rows, so the matrix kernels read straight
// 1 KB runs and never see a masked value.
#pragma once

#include <type_traits>

#include "attn.hpp"
#include "device_util.hpp"

namespace cgtp {
namespace attn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;  // 4 waves

// The kernels ask for two waves a SIMD, i.e. at most 256 registers a lane: their
// accumulators then sit in ordinary registers, where with a budget of 512 the
// compiler keeps them in the accumulation file and moves them to and fro for
// every vector operation (the forward of a head of 128 took 1.3 times as long).
// The heads whose whole tiles do not fit 256 registers take one wave.
constexpr int few_waves(int dp, size_t size) { return dp * int(size) <= (size == 2 ? 320 : 384) ? 2 : 1; }
// two workgroups a compute unit, where its 160 KB of shared memory hold `units` KB twice
constexpr int lds_waves(int units) { return units < 80 ? 2 : 1; }

// Matrix operands: 16 bytes a lane.
template <typename T>
struct Op;
template <>
struct Op<bf16> {
  static constexpr int VE = 8;
  using Frag = bf16x8;
  static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  // accumulator registers VE f .. VE f + 7 rounded to an operand
  static __device__ __forceinline__ Frag from_acc(const f32x16& s, int f) {
    Frag r;
#pragma unroll
    for (int j = 0; j < VE; ++j) r[j] = static_cast<__bf16>(s[VE * f + j]);
    return r;
  }
  // c + the sum of an operand's values (products with 1, summed in fp32)
  static __device__ __forceinline__ float add(Frag a, float c) {
    const bf16x2 one = {static_cast<__bf16>(1.0f), static_cast<__bf16>(1.0f)};
    const u32x4 v = __builtin_bit_cast(u32x4, a);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t pair = v[j];
      c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), one, c, false);
    }
    return c;
  }
};
template <>
struct Op<float> {
  static constexpr int VE = 4;
  using Frag = f32x4;
  static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ Frag from_acc(const f32x16& s, int f) {
    Frag r;
#pragma unroll
    for (int j = 0; j < VE; ++j) r[j] = s[VE * f + j];
    return r;
  }
};

template <typename T, int DP>
struct Dims {
  static constexpr int VE = Op<T>::VE;
  static constexpr int KSTEPS = DP / (2 * VE);  // row fragments of a tile
  static constexpr int DT = DP / 32;            // column groups of a tile
  static constexpr int FR = 16 / VE;            // column fragments of a column group
  static constexpr int TILE = DP * 32;          // elements of a packed tile
  static constexpr int UNITS = TILE * int(sizeof(T)) / 1024;
  // the widest heads (fp32, 256) leave too few registers for whole operands: some
  // are read again from memory as they are used
  static constexpr bool kShort = DP * int(sizeof(T)) > 896;
};

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}

// max and sum over the two halves of a wave (the two lanes of one query).
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// max over the lanes of a wave
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 1; off < 64; off *= 2) v = fmaxf(v, lane_fetch(v, (int(threadIdx.x & 63) ^ off) << 2));
  return v;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Unit u of a packed tile, this lane's 16 bytes.
template <typename T>
__device__ __forceinline__ u32x4 unit16(const T* tile, int u, int lane) {
  return *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(tile) + u * 1024 + lane * 16);
}
template <typename F>
__device__ __forceinline__ F as_frag(const u32x4& v) {
  return __builtin_bit_cast(F, v);
}

// One 1 KB unit copied from memory to shared memory without passing the
// registers; complete after wait_copies() and a barrier. dst is uniform over the
// wave.
template <typename T>
__device__ __forceinline__ void copy_unit(const T* tile, int u, int lane, u32x4* dst) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void*)(reinterpret_cast<const char*>(tile) + u * 1024 + lane * 16),
      (__attribute__((address_space(3))) void*)(dst), 16, 0, 0);
}
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// The end of a turn: all but the last N copies of this wave have arrived, its
// reads of shared memory are done, and the other waves have come as far. (Not
// __syncthreads(), which waits for every copy.)
template <int N>
__device__ __forceinline__ void turn_end() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// The lane, computed where it is needed (so that it holds no register meanwhile).
__device__ __forceinline__ int lane_id() {
  return int(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)));
}
// A value that is the same in all lanes, as a scalar.
__device__ __forceinline__ float uniform(float v) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 64); }

// Element address of head-vector element d of query row (token, head) or of
// context row (token, head): table entry (query offset, context offset,
// channels per head, 1 inside the head).
__device__ __forceinline__ int64_t elem(const int4& e, bool query, int head) {
  return (query ? e.x : e.y) + int64_t(head) * e.z;
}

// Rows are read without conditions: places outside the head have the table entry
// 0, i.e. the row's start, and are cleared when all loads are on their way (a
// condition around each would make every load wait for the one before).

// Pieces d0 = VE (first + 8 c) of a row, c = 0 .. PER - 1 (the last valid piece
// where there are fewer).
template <typename T, bool VEC, int PIECES, int PER>
__device__ __forceinline__ void load_pieces(const T* row, const int4* table, int first, bool query, int head,
                                            u32x4 (&v)[PER]) {
  constexpr int VE = Op<T>::VE;
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < PER; ++c)
      v[c] = *reinterpret_cast<const u32x4*>(row + elem(table[VE * min(first + 8 * c, PIECES - 1)], query, head));
  } else {
    T t[PER][VE];
#pragma unroll
    for (int c = 0; c < PER; ++c)
#pragma unroll
      for (int j = 0; j < VE; ++j) t[c][j] = row[elem(table[VE * min(first + 8 * c, PIECES - 1) + j], query, head)];
#pragma unroll
    for (int c = 0; c < PER; ++c) __builtin_memcpy(&v[c], t[c], 16);
  }
}

// The elements of piece d0 that lie inside a head of `size` elements.
template <typename T, bool VEC>
__device__ __forceinline__ u32x4 inside_head(u32x4 v, int d0, int size) {
  constexpr int VE = Op<T>::VE;
  if constexpr (VEC) return d0 < size ? v : u32x4{0, 0, 0, 0};
  if (d0 + VE > size) {
    T t[VE];
    __builtin_memcpy(t, &v, 16);
#pragma unroll
    for (int j = 0; j < VE; ++j)
      if (d0 + j >= size) t[j] = T{};
    __builtin_memcpy(&v, t, 16);
  }
  return v;
}

// Table entry d0 of the lower half of a wave, d0 + step of the upper one, by the
// scalar unit.
__device__ __forceinline__ int4 half_entry(const int4* table, int d0, int step, int h) {
  const int4 a = ldc(table + d0), b = ldc(table + d0 + step);
  return h ? b : a;
}

// Four consecutive head elements d0 .. d0 + 3 of one row, from fp32.
template <typename T>
__device__ __forceinline__ void scatter4(T* row, const int4* table, int d0, bool query, int head, bool quad,
                                         const float (&v)[4]) {
  const int4 e = table[d0];
  if (!e.w) return;
  if (quad) {
    VecIO<T, 4>::store(row + elem(e, query, head), v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int4 ej = table[d0 + j];
      if (ej.w) from_acc(row[elem(ej, query, head)], v[j]);
    }
  }
}

// A lane's part of a row (transposed accumulators g times scale): elements
// 8 b + 4 h .. + 3 of every column group.
template <typename T, int DT>
__device__ __forceinline__ void scatter_acc(T* row, const int4* table, bool query, int head, bool quad, int h,
                                            const f32x16 (&g)[DT], float scale) {
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = g[d][4 * b + i] * scale;
      if (quad) {
        const int4 e = half_entry(table, 32 * d + 8 * b, 4, h);
        if (e.w) VecIO<T, 4>::store(row + elem(e, query, head), v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int4 e = half_entry(table, 32 * d + 8 * b + i, 4, h);
          if (e.w) from_acc(row[elem(e, query, head)], v[i]);
        }
      }
    }
}

// ------------------------------------------------------------------ packing
//
// One workgroup packs one 32-row tile of one head group of both tensors of a
// call: 16-byte gathers, row fragments written straight from the registers that
// received them (a lane's piece of a row is a piece of a fragment), column
// fragments by way of shared memory. Bound: memory, each element read once and
// written once per form; both tensors' loads are issued together, since what
// holds a small workgroup up is the latency of its chain of loads.
//
// VEC: every tensor's runs are whole aligned 16-byte pieces (else read element by
// element); GRADS: the tensors are q and grad_out, with out for delta. As run-time
// arguments they cost registers, i.e. waves (ragged batch 615 us against 609 us; with
// unaligned rows 257 us against 232 us). A context of 32,764 rows of 4 KB packs at
// 3.8 TB/s read and written, one of 72,000 rows at 4.9 TB/s. Reading whole cache lines
// across neighbouring heads instead of one head's runs was no faster (155 us against
// 143 us): the lines are shared in the die's L2 already.
//
// CHECK: also notes the tiles that hold an infinity or NaN (redo_kernel).
template <typename T>
__device__ __forceinline__ bool not_finite(const u32x4& v) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bad = bad || (v[i] & 0x7f800000u) == 0x7f800000u;
    if (sizeof(T) == 2) bad = bad || (v[i] & 0x7f80u) == 0x7f80u;
  }
  return bad;
}
template <typename T, int DP, bool VEC, bool GRADS, bool CHECK = false>
__global__ __launch_bounds__(kThreads) void pack_kernel(PackArgs a) {
  using D = Dims<T, DP>;
  constexpr int VE = D::VE, LD = DP + VE;  // an odd count of 16-byte pieces a row: no bank conflicts
  constexpr int PIECES = DP / VE, PER = (PIECES + 7) / 8;
  // without GRADS one tensor at most has column fragments
  constexpr int B = GRADS ? 1 : 0;  // place of tensor 1
  __shared__ __attribute__((aligned(16))) T sh[B + 1][32 * LD];
  __shared__ float red[32][9];
  __shared__ int bad[CHECK ? 4 : 1];
  // A head's channels are short runs of a row: the heads of one tile share its
  // cache lines, so they go to one die (workgroup index modulo 8), one after another
  const int turn = int(blockIdx.x) / 8, tile = turn / a.groups * 8 + int(blockIdx.x) % 8, hk = turn % a.groups;
  if (tile >= a.ntiles) return;
  const Tile tl = ldc(a.tiles + tile);
  const int tid = int(threadIdx.x), lane = tid % 64, wave = wave_id();
  const bool query = a.G > 0;
  const int G = query ? a.G : 1;
  // 8 threads a row, every eighth piece each
  const int r = tid / 8;
  const bool in = r < tl.n;
  const int grow = tl.row0 + (in ? r : 0);
  const int token = grow / G, head = hk * G + grow % G;
  // masked rows, and queries and gradients of rows that saw nothing, count as zero
  const uint8_t seen = a.mask ? a.mask[token] : 1;
  const float lse = GRADS ? a.lse[int64_t(token) * a.heads + head] : 0.0f;
  // (rows that do not count are read as well: the mask need not be waited for)
  const auto row = [&](const void* src, int64_t ld) { return static_cast<const T*>(src) + int64_t(token) * ld; };
  u32x4 v0[PER], v1[PER], vo[PER];
  load_pieces<T, VEC, PIECES>(row(a.t[0].src, a.t[0].ld), a.table, tid % 8, query, head, v0);
  load_pieces<T, VEC, PIECES>(row(a.t[1].src, a.t[1].ld), a.table, tid % 8, query, head, v1);
  if constexpr (GRADS) load_pieces<T, VEC, PIECES>(row(a.out, a.ldo), a.table, tid % 8, query, head, vo);
  const bool live = in && seen != 0 && (!GRADS || lse != -INFINITY);
#pragma unroll
  for (int c = 0; c < PER; ++c) {
    const u32x4 none = {0, 0, 0, 0};
    const int d0 = VE * (tid % 8 + 8 * c);  // beyond the head where there is no such piece
    v0[c] = live ? inside_head<T, VEC>(v0[c], d0, a.size) : none;
    v1[c] = live ? inside_head<T, VEC>(v1[c], d0, a.size) : none;
    if constexpr (GRADS) vo[c] = live ? inside_head<T, VEC>(vo[c], d0, a.size) : none;
  }
  const int64_t at = int64_t(tile) * a.groups + hk;
  // piece p of row r is lane r + 32 (p % 2) of row fragment p / 2
  const auto rows = [&](const PackTensor& t, const u32x4 (&v)[PER]) {
    if (!t.row_frags) return;
    u32x4* o = reinterpret_cast<u32x4*>(static_cast<T*>(t.row_frags) + at * D::TILE);
#pragma unroll
    for (int c = 0; c < PER; ++c) {
      const int p = tid % 8 + 8 * c;
      if (PIECES % 8 != 0 && p >= PIECES) break;
      o[p / 2 * 64 + p % 2 * 32 + r] = v[c];
    }
  };
  rows(a.t[0], v0);
  rows(a.t[1], v1);
#pragma unroll
  for (int c = 0; c < PER; ++c) {
    const int d0 = (tid % 8 + 8 * c) * VE;
    if (PIECES % 8 != 0 && d0 >= DP) break;
    if (a.t[0].col_frags) *reinterpret_cast<u32x4*>(&sh[0][r * LD + d0]) = v0[c];
    if (a.t[1].col_frags) *reinterpret_cast<u32x4*>(&sh[B][r * LD + d0]) = v1[c];
  }
  if constexpr (CHECK) {
    bool found = false;
#pragma unroll
    for (int c = 0; c < PER; ++c) found = found || not_finite<T>(v0[c]) || not_finite<T>(v1[c]);
    const bool some = __any(found);
    if (lane == 0) bad[wave] = some;
  }
  if (!GRADS && a.norms) {
    // |k|^2 of every row, the largest of the tile below
    float n2 = 0.0f;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
      T tv[VE];
      __builtin_memcpy(tv, &v0[c], 16);
#pragma unroll
      for (int j = 0; j < VE; ++j) n2 += to_acc<float>(tv[j]) * to_acc<float>(tv[j]);
    }
    red[r][tid % 8] = n2;
  }
  if constexpr (GRADS) {
    float partial = 0.0f;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
      T tv[VE], to[VE];
      __builtin_memcpy(tv, &v1[c], 16);
      __builtin_memcpy(to, &vo[c], 16);
#pragma unroll
      for (int j = 0; j < VE; ++j) partial += to_acc<float>(tv[j]) * to_acc<float>(to[j]);
    }
    red[r][tid % 8] = partial;
  }
  __syncthreads();
  if constexpr (CHECK)
    if (tid == 0) a.bad[at] = bad[0] | bad[1] | bad[2] | bad[3];
  if (GRADS && tid % 8 == 0) {
    // log2-domain lse (+inf: the row contributes nothing; NaN stays: every weight of the
    // row is NaN then) and rowsum(grad_out out)
    float d = 0.0f;
    for (int k = 0; k < 8; ++k) d += red[r][k];
    a.rows_out[at * 64 + r] = in && lse != -INFINITY ? lse * 1.44269504088896341f : INFINITY;
    a.rows_out[at * 64 + 32 + r] = d;
  }
  if (!GRADS && a.norms && wave == 0) {
    float n2 = 0.0f;
    for (int k = 0; k < 8; ++k) n2 += red[lane % 32][k];
    const bool nan = __any(n2 != n2);
    n2 = wave_max(n2);
    if (lane == 0) a.norms[at] = nan ? INFINITY : n2;
  }
  if (!GRADS && a.bias && hk == 0 && tid < 32) {
    const bool seen = tid < tl.n && (a.mask == nullptr || a.mask[tl.row0 + tid] != 0);
    a.bias[int64_t(tile) * 32 + tid] = seen ? 0.0f : -INFINITY;
    const bool some = __any(!seen);
    if (a.flags && tid == 0) a.flags[tile] = some;
  }
  const int n = lane % 32, h = lane / 32;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!a.t[k].col_frags) continue;
    u32x4* o = reinterpret_cast<u32x4*>(static_cast<T*>(a.t[k].col_frags) + at * D::TILE);
    for (int u = wave; u < D::UNITS; u += 4) {
      const int dt = u / D::FR, f = u % D::FR;
      T t[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const int rr = VE * f + j;
        t[j] = sh[k * B][(8 * (rr / 4) + 4 * h + rr % 4) * LD + 32 * dt + n];
      }
      u32x4 v;
      __builtin_memcpy(&v, t, 16);
      o[u * 64 + lane] = v;
    }
  }
}

// ------------------------------------------------------------------- forward

// Running softmax of 32 queries: a lane holds its query's reference m (log2
// domain), its own keys' sum l of the weights as the matrix cores take them, and
// O^T. bf16 rounds the weights, and O / l is then still a mean of the values with
// weights that add up to one: a row that sees one key gives exactly its value,
// and its score gradients P (dP - delta) cancel. Where bf16 results come with the
// lse, the sum before rounding is formed beside l (from l the lse would be off by
// up to 2^-9).
template <int DT>
struct Running {
  float m = -INFINITY, l = 0.0f;
  f32x16 o[DT];
};

// The largest score of a lane's query in a tile (log2 domain; scale2 is positive,
// so the maximum is taken before scaling).
__device__ __forceinline__ float top_score(const f32x16& s, float scale2) {
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
  return half_max(mx) * scale2;
}

// Moves the reference up to a tile's top score. It follows only when that grows
// by more than 2^8: the weights stay below 2^8 (their sum is fp32), and most
// tiles need no rescaling of O.
template <int DT>
__device__ __forceinline__ void raise_reference(Running<DT>& st, float top, float& e, bool exact) {
  if (__any(top > st.m + 8.0f)) {
    const float mn = fmaxf(st.m, top);
    const float alpha = mn == -INFINITY ? 1.0f : exp2_fast(st.m - mn);
    st.m = mn;
    st.l *= alpha;
    if (exact) e *= alpha;
#pragma unroll
    for (int d = 0; d < DT; ++d) st.o[d] *= alpha;
  }
}

// Turns a tile's products q.k into weights exp2(scale2 q.k - m), the operands p;
// m is `fixed` unless MOVING.
template <typename T, bool MOVING, int DT>
__device__ __forceinline__ void weigh(Running<DT>& st, f32x16& s, float scale2, float fixed, float& e, bool exact,
                                      typename Op<T>::Frag (&p)[16 / Op<T>::VE]) {
  const float ref = !MOVING ? fixed : st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = exp2_fast(fmaf(s[i], scale2, -ref));
#pragma unroll
  for (int f = 0; f < 16 / Op<T>::VE; ++f) p[f] = Op<T>::from_acc(s, f);
  const auto add = [&](float& to) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += s[i];
    to += sum;
  };
  if constexpr (sizeof(T) == 2) {
    if (exact) add(e);
#pragma unroll
    for (int f = 0; f < 16 / Op<T>::VE; ++f) st.l = Op<T>::add(p[f], st.l);
  } else {
    add(st.l);
  }
}

// -inf for every masked or missing key of a tile (not by addition: the score of a
// NaN query is NaN for such keys too, and a row without a key is 0 whatever it holds).
__device__ __forceinline__ void mask_scores(f32x16& s, const float* bias, int h) {
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const f32x4 bv = *reinterpret_cast<const f32x4*>(bias + 8 * b + 4 * h);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[4 * b + i] = bv[i] < 0.0f ? -INFINITY : s[4 * b + i];
  }
}

// The key tile that tile t of a work list stands for.
template <bool SEQ, typename A>
__device__ __forceinline__ int key_tile(const A& a, int skip, int t) {
  return SEQ && t >= a.shared ? t + skip : t;
}

// Causal queries: a token's first hidden place among its own keys.
template <typename A>
__device__ __forceinline__ int hidden_from(const A& a, const Reach& re, int row) {
  return row / a.G + re.shift;
}

// -inf for the keys of a tile from place `hidden` on (replaced, not added to: see
// mask_scores).
__device__ __forceinline__ void hide_later(f32x16& s, int tile, int hidden, int h) {
  const int left = hidden - 32 * tile - 4 * h;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = 8 * (i / 4) + i % 4 < left ? s[i] : -INFINITY;
}

// Query fragments of tile `tl` straight from the rows.
template <typename T, int DP>
__device__ __forceinline__ void load_queries(const FwdArgs& a, const Tile& tl, int hk, int lane,
                                             typename Op<T>::Frag (&q)[Dims<T, DP>::KSTEPS]) {
  using D = Dims<T, DP>;
  const int n = lane % 32, h = lane / 32;
  const int row = tl.row0 + (n < tl.n ? n : tl.n - 1);
  const int token = row / a.G, head = hk * a.G + row % a.G;
  const T* src = static_cast<const T*>(a.q) + int64_t(token) * a.ldq;
  // a negative scale: the sign goes to the queries
  if (a.q_vec) {
    u32x4 v[D::KSTEPS];
#pragma unroll
    for (int t = 0; t < D::KSTEPS; ++t)
      v[t] = *reinterpret_cast<const u32x4*>(src + elem(half_entry(a.table, 2 * D::VE * t, D::VE, h), true, head));
#pragma unroll
    for (int t = 0; t < D::KSTEPS; ++t) {
      const u32x4 inside = half_entry(a.table, 2 * D::VE * t, D::VE, h).w ? v[t] : u32x4{0, 0, 0, 0};
      q[t] = as_frag<typename Op<T>::Frag>(inside ^ a.q_sign);
    }
  } else {
#pragma unroll
    for (int t = 0; t < D::KSTEPS; ++t) {
      T e[D::VE];
#pragma unroll
      for (int j = 0; j < D::VE; ++j) {
        const int4 at = half_entry(a.table, 2 * D::VE * t + j, D::VE, h);
        const T x = src[elem(at, true, head)];
        e[j] = at.w ? x : T{};
      }
      u32x4 v;
      __builtin_memcpy(&v, e, 16);
      q[t] = as_frag<typename Op<T>::Frag>(v ^ a.q_sign);
    }
  }
}

// With few registers left: keeps the scheduler from reading operands far ahead.
template <typename T, int DP>
__device__ __forceinline__ void pace(int u) {
  if (Dims<T, DP>::kShort && u % 4 == 3) __builtin_amdgcn_sched_barrier(0);
}

// Stages kept in shared memory: two where they fit, the next one on its way
// while this one is worked on, else one.
constexpr int stage_buffers(int units) { return 2 * units <= 152 ? 2 : 1; }
constexpr int stage_units(int units) { return stage_buffers(units) * units; }
// Tiles of a stage of dkv_kernel: Q rows, dO columns [grad_v], dO rows and Q
// columns [grad_k].
constexpr int dkv_forms(int part) { return part == 0 ? 4 : part == 1 ? 2 : 3; }

// Writes a wave's result: final rows, or an unnormalised part of a split (of
// `part_rows` rows a tile).
template <typename T, int DP>
__device__ __forceinline__ void finish(const FwdArgs& a, const Item& it, const Tile& tl, int tile_in_item,
                                       const Running<DP / 32>& st, float exact_sum, int part_rows = 32) {
  const int lane = lane_id(), n = lane % 32, h = lane / 32;
  const float l = half_sum(st.l), e = sizeof(T) == 2 ? half_sum(exact_sum) : l;
  if (n >= tl.n) return;
  if (it.slot >= 0) {
    const int64_t r = (int64_t(it.slot) * it.stride + tile_in_item) * part_rows + n;
    float* o = a.part + r * DP;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = st.o[d][4 * b + i];
        *reinterpret_cast<f32x4*>(o + 32 * d + 8 * b + 4 * h) = v;
      }
    // (a part without a visible key has no reference: that of bounded scores would
    // stand above those of the other parts when they are joined)
    if (h == 0) a.part_ml[r] = make_float4(l == 0.0f ? -INFINITY : st.m, l, e, 0.0f);
    return;
  }
  const int row = tl.row0 + n, token = row / a.G, head = it.hk * a.G + row % a.G;
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  scatter_acc(static_cast<T*>(a.out) + int64_t(token) * a.ldo, a.table, true, head, a.out_quad, h, st.o, inv);
  if (a.lse && h == 0)
    a.lse[int64_t(token) * a.heads + head] = l > 0.0f || l != l ? (st.m + __log2f(e)) * 0.69314718055994531f : -INFINITY;
}

// The kernel's arguments (its only parameter) read anew: what a branch that is hardly ever
// taken needs of them would else be held in registers, or spilled, by all that comes before.
template <typename A>
__device__ __forceinline__ const A& arguments_anew() {
  auto p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const A*)(p);
}

// Lanes whose accumulators hold a NaN.
template <int DT>
__device__ __forceinline__ bool any_nan(const f32x16 (&o)[DT]) {
  bool nan = false;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) nan = nan || o[d][i] != o[d][i];
  return nan;
}
// The rows (lanes modulo 32) for which `bad` holds in either half.
__device__ __forceinline__ uint32_t rows_of(bool bad) {
  const uint64_t b = __ballot(bad);
  return uint32_t(b) | uint32_t(b >> 32);
}

// A matrix product adds weight 0 times what a row does not see, which is NaN where that is
// infinite or NaN. Rows that this reaches are formed again with products that leave it out
// (redo_rows, redo_kernel): infinities and NaN go into the product as 1 with their sign, and what
// they add to a result is counted beside it by two more products, a of the signs of the infinities
// and of the weights, b of the infinities and NaN and the rows that see them. Where b = 0 there are
// none; where |a| = b all are infinities that add one sign; else there is a NaN among them,
// or infinities of both signs or with weight 0. Both counts are at most 32 a tile and kept as a + 128 b.
// Everything here is on a branch that is hardly ever taken, so it takes 32 columns of a head at a time, with
// all products of the scores again for each: its registers must not cost the kernels around it their
// waves (all columns at once: 156 for heads of 32 in bf16, where the forward has 76).

// The weights of a tile (0 where not seen) as operands.
template <typename T>
struct SeenWeights {
  static constexpr int VE = Op<T>::VE, FR = 16 / VE;
  using Frag = typename Op<T>::Frag;
  Frag w[FR];
  uint32_t seen;  // bit i: the row sees what accumulator register i stands for
  __device__ __forceinline__ float sign(int f, int j) const {
    const float x = static_cast<float>(w[f][j]);
    return x > 0.0f ? 1.0f : x < 0.0f ? -1.0f : 0.0f;
  }
  __device__ __forceinline__ float one(int f, int j) const { return float(seen >> (VE * f + j) & 1); }
};
// acc += columns 32 d .. of a packed tile times weights, of seen pairs alone.
template <typename T>
__device__ __forceinline__ void add_seen(f32x16& acc, const T* columns, int d, const SeenWeights<T>& s) {
  constexpr int VE = Op<T>::VE, FR = 16 / VE;
  using Frag = typename Op<T>::Frag;
  using E = std::remove_reference_t<decltype(Frag{}[0])>;
  bool bad = false;
#pragma unroll
  for (int f = 0; f < FR; ++f) {
    const u32x4 bits = unit16(columns, d * FR + f, lane_id());
    bad = bad || not_finite<T>(bits);
    Frag x = as_frag<Frag>(bits);
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const float v = static_cast<float>(x[j]);
      x[j] = fabsf(v) < INFINITY ? x[j] : static_cast<E>(copysignf(1.0f, v));
    }
    acc = Op<T>::mma(x, s.w[f], acc);
    __builtin_amdgcn_sched_barrier(0);
  }
  if (!__any(bad)) return;
  f32x16 count = zero16();
#pragma unroll
  for (int f = 0; f < FR; ++f) {
    const Frag x = as_frag<Frag>(unit16(columns, d * FR + f, lane_id()));
    Frag y, w;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const float v = static_cast<float>(x[j]);
      y[j] = static_cast<E>(fabsf(v) == INFINITY ? copysignf(1.0f, v) : 0.0f);
      w[j] = static_cast<E>(s.sign(f, j));
    }
    count = Op<T>::mma(y, w, count);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      y[j] = static_cast<E>(fabsf(static_cast<float>(x[j])) < INFINITY ? 0.0f : 128.0f);
      w[j] = static_cast<E>(s.one(f, j));
    }
    count = Op<T>::mma(y, w, count);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float b = rintf(count[i] * 0.0078125f), a = count[i] - 128.0f * b;
    acc[i] += b == 0.0f ? 0.0f : fabsf(a) == b ? copysignf(INFINITY, a) : NAN;
  }
}
// Bits of a lane's accumulator registers whose places, of the 32 from `first` on, lie below `end`.
__device__ __forceinline__ uint32_t seen_below(int first, int end, int h) {
  uint32_t seen = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) seen |= (first + 8 * (i / 4) + 4 * h + i % 4 < end ? 1u : 0u) << i;
  return seen;
}
// Elements 32 d + 8 b + 4 h .. + 3 of a lane's row from accumulators g times scale (as scatter_acc).
template <typename T>
__device__ __forceinline__ void scatter_columns(T* row, const int4* table, bool query, int head, int h, int d,
                                                const f32x16& g, float scale) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int4 e = table[32 * d + 8 * (i / 4) + 4 * h + i % 4];
    if (e.w) from_acc(row[elem(e, query, head)], g[i] * scale);
    if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
  }
}
__device__ __forceinline__ void store_columns(float* o, int h, const f32x16& g, float scale) {
#pragma unroll
  for (int b = 0; b < 4; ++b)
    *reinterpret_cast<f32x4*>(o + 8 * b + 4 * h) =
        f32x4{g[4 * b] * scale, g[4 * b + 1] * scale, g[4 * b + 2] * scale, g[4 * b + 3] * scale};
}

// Rows of a causal forward that came out NaN with a finite sum of weights, where values in
// tiles that some of the rows see only a part of may be why: formed again after finish() wrote
// them, with the reference that they had, from the wave's tiles in memory (1500 rows, 4 heads of
// 128, one NaN among the values: 89 us for 42 in bf16, 187 us for 63 in fp32; NaN in all of
// them 142 and 216 us).
template <typename T, int DP>
__device__ __forceinline__ void redo_rows(const Item& it, const Reach& re, const Tile& tl, int tile_in_item,
                                          const Running<DP / 32>& st) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  const float sum = half_sum(st.l);
  const uint32_t rows = rows_of(any_nan(st.o) && sum == sum);
  if (!rows) return;
  const FwdArgs& a = arguments_anew<FwdArgs>();
  const int lane = lane_id(), n = lane % 32, h = lane / 32;
  const auto tile_of = [&](const void* src, int tile) {
    return static_cast<const T*>(src) + (int64_t(tile) * a.groups + it.hk) * D::TILE;
  };
  bool bad = false;
  const int part = hidden_from(a, re, tl.row0) >> 5;
  for (int t = it.b1 - 1; t >= max(it.b0, a.shared); --t) {
    const int tile = key_tile<true>(a, re.skip, t);
    if (tile < part) break;
#pragma unroll 1
    for (int u = 0; u < D::UNITS; ++u) bad = bad || not_finite<T>(unit16(tile_of(a.vf, tile), u, lane));
  }
  if (!__any(bad)) return;
  wait_copies();  // (finish's stores of the same rows come first)
  const int row = tl.row0 + min(n, tl.n - 1), token = row / a.G, head = it.hk * a.G + row % a.G;
  const int hidden = hidden_from(a, re, row);
  const bool mine = n < tl.n && (rows >> n & 1);
  const float m = st.m;
#pragma unroll 1
  for (int d = 0; d < D::DT; ++d) {
    Running<1> again;
    float e = 0.0f;
    again.m = m;
    again.o[0] = zero16();
#pragma unroll 1
    for (int t = it.b0; t < it.b1; ++t) {
      const int tile = key_tile<true>(a, re.skip, t);
      f32x16 s = zero16();
      {
        Frag q[D::KSTEPS];
        load_queries<T, DP>(a, tl, it.hk, lane, q);
#pragma unroll
        for (int u = 0; u < D::KSTEPS; ++u) {
          s = Op<T>::mma(as_frag<Frag>(unit16(tile_of(a.kf, tile), u, lane)), q[u], s);
          if (u % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (ldc(a.flags + tile)) mask_scores(s, a.bias + int64_t(tile) * 32, h);
      SeenWeights<T> x;
      x.seen = t < a.shared ? 0xffffu : seen_below(32 * tile, hidden, h);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = x.seen >> i & 1 ? s[i] : -INFINITY;
      weigh<T, true>(again, s, a.scale2, 0.0f, e, false, x.w);
      __builtin_amdgcn_sched_barrier(0);
      add_seen(again.o[0], tile_of(a.vf, tile), d, x);
    }
    const float l = half_sum(again.l);
    if (!mine) continue;
    if (it.slot >= 0) {
      const int64_t r = (int64_t(it.slot) * it.stride + tile_in_item) * 32 + n;
      store_columns(a.part + r * DP + 32 * d, h, again.o[0], 1.0f);
      if (h == 0) a.part_ml[r].y = l;  // (reference and exact sum stay)
    } else {
      scatter_columns(static_cast<T*>(a.out) + int64_t(token) * a.ldo, a.table, true, head, h, d, again.o[0],
                      l > 0.0f || l != l ? 1.0f / l : 0.0f);
    }
  }
}

// Tiles of the keys and of the values in shared memory: R - 1 turns for a copy to
// arrive. Three where that leaves room for two workgroups a compute unit (long
// contexts, head of 128: 1153 us, with two 1159 us).
template <typename T, int DP>
constexpr int fwd_ring() {
  return 6 * Dims<T, DP>::UNITS < 80 ? 3 : 2;
}

// The square of a bound of all scores (log2 domain) of a wave's queries against
// the tiles of an item: |q.k| <= |q| |k|. NaN where a row holds one.
template <typename T, int DP, int RT, bool SEQ>
__device__ __forceinline__ float score_bound2(const FwdArgs& a, const Item& it, int skip, int lane,
                                              const typename Op<T>::Frag (&q)[RT][Dims<T, DP>::KSTEPS]) {
  using D = Dims<T, DP>;
  float qn = 0.0f, kn = 0.0f;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float n2 = 0.0f;
#pragma unroll
    for (int u = 0; u < D::KSTEPS; ++u)
#pragma unroll
      for (int j = 0; j < D::VE; ++j) {
        const float e = static_cast<float>(q[r][u][j]);
        n2 += e * e;
      }
    n2 = half_sum(n2);
    qn = n2 > qn || n2 != n2 ? n2 : qn;
  }
  for (int t = it.b0 + lane; t < it.b1; t += 64) {
    const float n2 = a.norms[int64_t(key_tile<SEQ>(a, skip, t)) * a.groups + it.hk];
    kn = n2 > kn || n2 != n2 ? n2 : kn;
  }
  const bool nan = __any(qn != qn || kn != kn);
  return nan ? INFINITY : wave_max(qn) * wave_max(kn) * a.scale2 * a.scale2;
}

// Scores bounded by B <= kBound (log2 domain) need no running maximum: with the
// reference max(B - 8, 0) their weights are at most 2^8, as with a running maximum, so
// that values as large as there can be summed, and the largest of a row is at least
// 2^(8 - 2 kBound) = 2^-72: its products with values above 2^-54 are normal numbers of
// fp32 (whose exponent range bf16 shares).
constexpr float kBound = 40.0f;

// Four waves of RT x 32 query rows share the keys through shared memory; the tiles
// of the next turns are on their way there while one is worked on. Bound: matrix
// cores, vector units (16 exponentials a lane and tile) and shared memory
// together; RT = 2 halves the operand reads from shared memory per product,
// which with the copies into it take 1.5 times as long as the products else. Two
// paths: scores bounded beforehand by the rows' norms (what normalised features
// give) go without maximum, branch and rescaling; others keep a running maximum
// (for RT = 2 one 32-row half after the other; long contexts, head of 128: 1068 us
// bounded, 1257 us with it).
// Measured: 4 x 4096 queries against 8191 keys, 16 heads of 128, bf16: 934 us =
// 1177 TFLOP/s (994 us over the first 50 passes of an idle card) with matrix cores busy
// 56 % of the cycles; a ragged batch of heads of 144 (RT = 1): 144 us, 30 %; fp32, heads of
// 128: 66 %.
//
// SEQ: key tiles by way of the queries' Reach, and in causal batches the scores of
// later keys hidden in the tiles where some of the wave's queries see only a part (one
// or two of a wave's; a wave leaves out the tiles that none of its queries sees).
template <typename T, int DP, int RT>
struct FwdShared {
  u32x4 kb[fwd_ring<T, DP>()][Dims<T, DP>::UNITS * 64], vb[fwd_ring<T, DP>()][Dims<T, DP>::UNITS * 64];
  float bounds[4], sums[sizeof(T) == 2 ? RT : 1][kThreads];
};
template <typename T, int DP, int RT, bool SEQ>
__device__ __forceinline__ void fwd_body(const FwdArgs& a, int item, FwdShared<T, DP, RT>& sh) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  constexpr int R = fwd_ring<T, DP>();
  auto& kb = sh.kb;
  auto& vb = sh.vb;
  auto& bounds = sh.bounds;
  auto& sums = sh.sums;
  const Item it = ldc(a.items + item);
  if (it.tiles == 0) return;
  const int lane = int(threadIdx.x) % 64, wave = wave_id(), h = lane / 32;
  const int mine = min(max(it.tiles - wave * RT, 0), RT);  // query tiles of this wave
  const int n = it.b1 - it.b0;
  const Reach re = SEQ ? ldc(a.reach + it.a0) : Reach{0, 0};  // (all query tiles of an item are of one sample)
  // tile t of the keys and of the values, a quarter by each wave
  const auto copy = [&](int t, int slot) {
    const int64_t at = (int64_t(key_tile<SEQ>(a, re.skip, min(it.b0 + t, it.b1 - 1))) * a.groups + it.hk) * D::TILE;
#pragma unroll
    for (int k = 0; k < D::UNITS / 2; ++k) {
      const int u = k * 4 + wave;
      if (u < D::UNITS) copy_unit(static_cast<const T*>(a.kf) + at, u, lane, &kb[slot][u * 64]);
      else copy_unit(static_cast<const T*>(a.vf) + at, u - D::UNITS, lane, &vb[slot][(u - D::UNITS) * 64]);
    }
  };
  if (n > 0)
#pragma unroll
    for (int t = 0; t + 1 < R; ++t) copy(t, t);
  // a lane's own entry for each of its queries: no register to spare for it where RT = 2
  const bool exact = sizeof(T) == 2 && a.lse != nullptr;
  const auto sum = [&](int r) -> float& { return sums[sizeof(T) == 2 ? r : 0][threadIdx.x]; };
  Frag q[RT][D::KSTEPS];
  Running<D::DT> st[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    sum(r) = 0.0f;
    load_queries<T, DP>(a, ldc(a.qtiles + it.a0 + (r < mine ? wave * RT + r : 0)), it.hk, lane, q[r]);
#pragma unroll
    for (int d = 0; d < D::DT; ++d) st[r].o[d] = zero16();
  }
  // causal: own key tiles from `part` on hold keys that some query of a row of tiles does
  // not see, those from `none` on are seen by no query of the wave
  int part[RT], none = INT_MAX;
  if constexpr (SEQ)
    if (a.causal) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const Tile tl = ldc(a.qtiles + it.a0 + (r < mine ? wave * RT + r : 0));
        part[r] = hidden_from(a, re, tl.row0) >> 5;
        const int end = (hidden_from(a, re, tl.row0 + tl.n - 1) + 31) >> 5;
        none = r == 0 ? end : max(none, end);
      }
    }
  const float b2 = score_bound2<T, DP, RT, SEQ>(a, it, re.skip, lane, q);
  if (lane == 0) bounds[wave] = b2;
  turn_end<0>();
  bool bounded = true;
#pragma unroll
  for (int w = 0; w < 4; ++w) bounded = bounded && bounds[w] <= kBound * kBound;
  const float fixed = uniform(fmaxf(__builtin_amdgcn_sqrtf(b2) - 8.0f, 0.0f));  // the wave's reference, if bounded

  // A wave at its products goes before one at its exponentials, which then fill the
  // gaps (long contexts, head of 128: 1074 us against 1093 us; with 32 rows a wave the
  // products are too short for it: ragged batch of heads of 144 617 us against 610 us)
  const auto products = [](bool now) {
    if constexpr (RT == 2) {
      if (now) __builtin_amdgcn_s_setprio(1);
      else __builtin_amdgcn_s_setprio(0);
    }
  };
  // query tiles R0 .. R0 + N - 1 of every wave over all keys; tiles 0 .. R - 2 are there
  const auto run = [&](auto first, auto count, auto moving) {
    constexpr int R0 = decltype(first)::value, N = decltype(count)::value;
    constexpr bool kMoving = decltype(moving)::value;
    int slot = 0;
    for (int t = 0; t < n; ++t) {
      const int tile = key_tile<SEQ>(a, re.skip, it.b0 + t);
      const bool later = SEQ && a.causal && it.b0 + t >= a.shared;
      copy(t + R - 1, slot == 0 ? R - 1 : slot - 1);
      if (mine > R0 && !(later && tile >= none)) {
        f32x16 s[N];
        products(true);
#pragma unroll
        for (int r = 0; r < N; ++r) s[r] = zero16();
#pragma unroll
        for (int u = 0; u < D::KSTEPS; ++u) {
          const Frag kf = as_frag<Frag>(kb[slot][u * 64 + lane]);
#pragma unroll
          for (int r = 0; r < N; ++r) s[r] = Op<T>::mma(kf, q[R0 + r][u], s[r]);
        }
        products(false);
        if (ldc(a.flags + tile))
#pragma unroll
          for (int r = 0; r < N; ++r) mask_scores(s[r], a.bias + int64_t(tile) * 32, h);
        if constexpr (SEQ)
          if (later)
#pragma unroll
            for (int r = 0; r < N; ++r)
              if (tile >= part[R0 + r]) {
                const Tile tl = ldc(a.qtiles + it.a0 + (R0 + r < mine ? wave * RT + R0 + r : 0));
                hide_later(s[r], tile, hidden_from(a, re, tl.row0 + min(lane_id() % 32, tl.n - 1)), h);
              }
        Frag p[N][D::FR];
#pragma unroll
        for (int r = 0; r < N; ++r) {
          if (kMoving) raise_reference(st[R0 + r], top_score(s[r], a.scale2), sum(R0 + r), exact);
          weigh<T, kMoving>(st[R0 + r], s[r], a.scale2, fixed, sum(R0 + r), exact, p[r]);
        }
        products(true);
#pragma unroll
        for (int d = 0; d < D::DT; ++d)
#pragma unroll
          for (int f = 0; f < D::FR; ++f) {
            const Frag vf = as_frag<Frag>(vb[slot][(d * D::FR + f) * 64 + lane]);
#pragma unroll
            for (int r = 0; r < N; ++r) st[R0 + r].o[d] = Op<T>::mma(vf, p[r][f], st[R0 + r].o[d]);
          }
      }
      products(false);
      slot = slot + 1 == R ? 0 : slot + 1;
      turn_end<(R - 2) * D::UNITS / 2>();
    }
    wait_copies();  // none may land after the workgroup's end
    if (!kMoving)
#pragma unroll
      for (int r = R0; r < R0 + N; ++r) st[r].m = fixed;
  };
  using zero = std::integral_constant<int, 0>;
  using one = std::integral_constant<int, 1>;
  if (n > 0) {
    if (bounded) {
      run(zero{}, std::integral_constant<int, RT>{}, std::false_type{});
    } else {
      run(zero{}, one{}, std::true_type{});
      if constexpr (RT == 2) {
        __syncthreads();
#pragma unroll
        for (int t = 0; t + 1 < R; ++t) copy(t, t);
        turn_end<0>();
        run(one{}, one{}, std::true_type{});
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
    if (r < mine) {
      const Tile tl = ldc(a.qtiles + it.a0 + wave * RT + r);
      finish<T, DP>(a, it, tl, wave * RT + r, st[r], sum(r));
      if constexpr (SEQ)
        if (a.causal) redo_rows<T, DP>(it, re, tl, wave * RT + r, st[r]);
    }
}

template <typename T, int DP, int RT, bool SEQ>
__global__ __launch_bounds__(kThreads, lds_waves(2 * fwd_ring<T, DP>() * Dims<T, DP>::UNITS)) void fwd_kernel(
    FwdArgs a) {
  __shared__ FwdShared<T, DP, RT> sh;
  fwd_body<T, DP, RT, SEQ>(a, int(blockIdx.x), sh);
}

// At most 32 query rows against a long context (single tokens): the four waves
// take every fourth key tile, read straight into registers, and join. Bound: the
// keys' and values' bytes: 64 tokens against 1000 - 8000 keys each, heads of 128,
// bf16: 114 us = 5.4 TB/s.
template <typename T, int DP, bool SEQ>
__global__ __launch_bounds__(kThreads, few_waves(DP, sizeof(T))) void fwd_few_kernel(FwdArgs a) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  __shared__ f32x4 sh[2][D::DT * 4 * 64];
  __shared__ float ml[4][3][64];
  const Item it = ldc(a.items + blockIdx.x);
  if (it.tiles == 0) return;
  const int lane = int(threadIdx.x) % 64, wave = wave_id(), h = lane / 32;
  const Tile tl = ldc(a.qtiles + it.a0);
  const Reach re = SEQ ? ldc(a.reach + it.a0) : Reach{0, 0};
  // the widest heads leave no registers for whole tiles: read as they are used
  constexpr bool kStream = DP * int(sizeof(T)) > 640;
  // a tile's units, in registers a turn ahead: the keys' are read again as soon as
  // the scores are done, the values' as soon as they are added
  u32x4 k[kStream ? 1 : D::UNITS], v[kStream ? 1 : D::UNITS];
  const auto tile = [&](const void* src, int t) {
    return static_cast<const T*>(src) +
           (int64_t(key_tile<SEQ>(a, re.skip, min(t, it.b1 - 1))) * a.groups + it.hk) * D::TILE;
  };
  const auto fetch = [&](const T* src, auto& dst) {
    if constexpr (!kStream)
#pragma unroll
      for (int u = 0; u < D::UNITS; ++u) dst[u] = unit16(src, u, lane);
  };
  if (it.b0 + wave < it.b1) {
    fetch(tile(a.kf, it.b0 + wave), k);
    fetch(tile(a.vf, it.b0 + wave), v);
  }
  Frag q[D::KSTEPS];
  load_queries<T, DP>(a, tl, it.hk, lane, q);
  Running<D::DT> st;
  float e = 0.0f;
  const bool exact = sizeof(T) == 2 && a.lse != nullptr;
#pragma unroll
  for (int d = 0; d < D::DT; ++d) st.o[d] = zero16();
  for (int t = it.b0 + wave; t < it.b1; t += 4) {
    f32x16 sc = zero16();
#pragma unroll
    for (int u = 0; u < D::KSTEPS; ++u) {
      if constexpr (kStream) {
        sc = Op<T>::mma(as_frag<Frag>(unit16(tile(a.kf, t), u, lane)), q[u], sc);
        if (u % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      } else {
        sc = Op<T>::mma(as_frag<Frag>(k[u]), q[u], sc);
      }
    }
    fetch(tile(a.kf, t + 4), k);
    const int at = key_tile<SEQ>(a, re.skip, t);
    if (ldc(a.flags + at)) mask_scores(sc, a.bias + int64_t(at) * 32, h);
    if constexpr (SEQ)
      if (a.causal && t >= a.shared && at >= hidden_from(a, re, tl.row0) >> 5)
        hide_later(sc, at, hidden_from(a, re, tl.row0 + min(lane % 32, tl.n - 1)), h);
    raise_reference(st, top_score(sc, a.scale2), e, exact);
    Frag p[D::FR];
    weigh<T, true>(st, sc, a.scale2, 0.0f, e, exact, p);
#pragma unroll
    for (int d = 0; d < D::DT; ++d)
#pragma unroll
      for (int f = 0; f < D::FR; ++f) {
        const int u = d * D::FR + f;
        if constexpr (kStream) {
          st.o[d] = Op<T>::mma(as_frag<Frag>(unit16(tile(a.vf, t), u, lane)), p[f], st.o[d]);
          if (u % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        } else {
          st.o[d] = Op<T>::mma(as_frag<Frag>(v[u]), p[f], st.o[d]);
        }
      }
    fetch(tile(a.vf, t + 4), v);
  }
  // join: common reference, then waves 2, 3 into 0, 1 and 1 into 0
  ml[wave][0][lane] = st.m;
  __syncthreads();
  float m = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) m = fmaxf(m, ml[w][0][lane]);
  const float f = m == -INFINITY ? 1.0f : exp2_fast(st.m - m);
  st.m = m;
  st.l *= f;
  e *= f;
#pragma unroll
  for (int d = 0; d < D::DT; ++d) st.o[d] *= f;
  ml[wave][1][lane] = st.l;
  ml[wave][2][lane] = e;
#pragma unroll
  for (int round = 2; round >= 1; --round) {
    // the upper `round` waves write, the lower ones add
    if (wave >= round && wave < 2 * round)
#pragma unroll
      for (int d = 0; d < D::DT; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          f32x4 v;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = st.o[d][4 * b + i];
          sh[wave - round][(d * 4 + b) * 64 + lane] = v;
        }
    __syncthreads();
    if (wave < round)
#pragma unroll
      for (int d = 0; d < D::DT; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const f32x4 v = sh[wave][(d * 4 + b) * 64 + lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) st.o[d][4 * b + i] += v[i];
        }
    __syncthreads();
  }
  if (wave == 0) {
    st.l = ml[0][1][lane] + ml[2][1][lane] + (ml[1][1][lane] + ml[3][1][lane]);
    e = ml[0][2][lane] + ml[2][2][lane] + (ml[1][2][lane] + ml[3][2][lane]);
    finish<T, DP>(a, it, tl, 0, st, e);
    if constexpr (SEQ)
      if (a.causal) redo_rows<T, DP>(it, re, tl, 0, st);
  }
}

// Joins the parts of split rows: a workgroup takes 32 rows x 32 columns (columns
// of workgroup y), a thread 4 of them. Bound: the parts' bytes; the loads of all
// parts are independent, so they overlap.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void fwd_join_kernel(FwdArgs a) {
  const Join j = ldc(a.joins + blockIdx.x);
  const Tile tl = ldc(a.qtiles + j.tile);
  const int n = int(threadIdx.x) / 8, d = int(blockIdx.y) * 32 + int(threadIdx.x) % 8 * 4;
  if (n >= tl.n) return;
  const int64_t first = (int64_t(j.slot) * j.stride + j.within) * 32 + n, step = int64_t(j.stride) * 32;
  float m = -INFINITY, l = 0.0f, e = 0.0f;
#pragma unroll 4
  for (int k = 0; k < j.parts; ++k) m = fmaxf(m, a.part_ml[first + k * step].x);
  const float ref = m == -INFINITY ? 0.0f : m;
  float v[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int k = 0; k < j.parts; ++k) {
    const int64_t r = first + k * step;
    const float4 ml = a.part_ml[r];
    const float w = exp2_fast(ml.x - ref);
    l += ml.y * w;
    e += ml.z * w;
    const f32x4 o = *reinterpret_cast<const f32x4*>(a.part + r * DP + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += w * o[i];
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  const int row = tl.row0 + n, token = row / a.G, head = j.hk * a.G + row % a.G;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] *= inv;
  scatter4(static_cast<T*>(a.out) + int64_t(token) * a.ldo, a.table, d, true, head, a.out_quad, v);
  if (a.lse && d == 0)
    a.lse[int64_t(token) * a.heads + head] = l > 0.0f || l != l ? (ref + __log2f(e)) * 0.69314718055994531f : -INFINITY;
}

// ------------------------------------------------------------------ backward

// A wave's 32 x DP gradient (transposed accumulators): final rows or a part.
template <typename T, int DP>
__device__ __forceinline__ void finish_grad(const BwdArgs& a, const Item& it, const Tile& tl, int within, int lane,
                                            bool query, void* dst, int64_t ld, float* part, bool quad,
                                            const f32x16 (&g)[DP / 32], float scale) {
  const int n = lane % 32, h = lane / 32;
  if (it.slot >= 0) {
    float* o = part + ((int64_t(it.slot) * it.stride + within) * 32 + n) * DP;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = g[d][4 * b + i] * scale;
        *reinterpret_cast<f32x4*>(o + 32 * d + 8 * b + 4 * h) = v;
      }
    return;
  }
  if (n >= tl.n) return;
  const int row = tl.row0 + n, G = query ? a.G : 1, token = row / G, head = it.hk * G + row % G;
  scatter_acc(static_cast<T*>(dst) + int64_t(token) * ld, a.table, query, head, quad, h, g, scale);
}

// grad_q: as the forward, a wave keeps 32 query rows and walks the key tiles:
// S^T = K Q^T, P^T = exp2(S^T - lse), dP^T = V dO^T, dS^T = P^T (dP^T - delta),
// dQ^T += K^T dS^T. Three packed forms of a tile pass through shared memory: K
// rows, V rows, K columns.
template <typename T, int DP, bool SEQ>
__device__ __forceinline__ void dq_item(const BwdArgs& a, const Item& it, u32x4* pool, float* bias_pool) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  constexpr int STAGE = 3 * D::UNITS, PER = (STAGE + 3) / 4;
  constexpr int BUFS = stage_buffers(STAGE);
  const auto sh = reinterpret_cast<u32x4(*)[STAGE * 64]>(pool);
  const auto bias = reinterpret_cast<float(*)[64]>(bias_pool);
  const int lane = int(threadIdx.x) % 64, wave = wave_id(), n = lane % 32, h = lane / 32;
  const bool active = wave < it.tiles;
  const int qt = it.a0 + (active ? wave : 0);
  const Tile tl = ldc(a.qtiles + qt);
  const int64_t qat = int64_t(qt) * a.groups + it.hk;
  const T* const qrows = a.qforms<T>(kQRows) + qat * D::TILE;
  Frag q[D::kShort ? 1 : D::KSTEPS], g[D::KSTEPS];
#pragma unroll
  for (int t = 0; t < D::KSTEPS; ++t) {
    if constexpr (!D::kShort) q[t] = as_frag<Frag>(unit16(qrows, t, lane));
    g[t] = as_frag<Frag>(unit16(a.qforms<T>(kGRows) + qat * D::TILE, t, lane));
  }
  const float lse2 = a.rows[qat * 64 + n], delta = a.rows[qat * 64 + 32 + n];
  const Reach re = SEQ ? ldc(a.reach + qt) : Reach{0, 0};
  // causal: as in fwd_kernel
  int hidden = 0, part = 0, none = 0;
  if constexpr (SEQ)
    if (a.causal) {
      hidden = hidden_from(a, re, tl.row0 + min(n, tl.n - 1));
      part = hidden_from(a, re, tl.row0) >> 5;
      none = (hidden_from(a, re, tl.row0 + tl.n - 1) + 31) >> 5;
    }
  f32x16 dq[D::DT];
#pragma unroll
  for (int d = 0; d < D::DT; ++d) dq[d] = zero16();

  const auto fetch = [&](int t, int buf) {
    const int tile = key_tile<SEQ>(a, re.skip, t);
    const T* base = a.kforms<T>(0) + (int64_t(tile) * a.groups + it.hk) * D::TILE;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int u = k * 4 + wave, form = u / D::UNITS;
      if (u >= STAGE) break;
      copy_unit(base + form * a.kstride, u % D::UNITS, lane, &sh[buf][u * 64]);
    }
    if (threadIdx.x < 32) bias[buf][threadIdx.x] = a.bias[int64_t(tile) * 32 + threadIdx.x];
  };
  if (it.b0 < it.b1) fetch(it.b0, 0);
  wait_copies();
  __syncthreads();
  for (int t = it.b0; t < it.b1; ++t) {
    const int buf = BUFS == 2 ? (t - it.b0) & 1 : 0;
    if (BUFS == 2 && t + 1 < it.b1) fetch(t + 1, buf ^ 1);
    const int tile = key_tile<SEQ>(a, re.skip, t);
    const bool later = SEQ && a.causal && t >= a.shared;
    if (active && !(later && tile >= none)) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int u = 0; u < D::KSTEPS; ++u) {
        const Frag qu = D::kShort ? as_frag<Frag>(unit16(qrows, u, lane)) : q[D::kShort ? 0 : u];
        s = Op<T>::mma(as_frag<Frag>(sh[buf][u * 64 + lane]), qu, s);
        dp = Op<T>::mma(as_frag<Frag>(sh[buf][(D::UNITS + u) * 64 + lane]), g[u], dp);
        pace<T, DP>(u);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f32x4 bv = *reinterpret_cast<const f32x4*>(&bias[buf][8 * b + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = exp2_fast(fmaf(s[4 * b + i], a.scale2, bv[i]) - lse2);
          s[4 * b + i] = p * (dp[4 * b + i] - delta);
        }
      }
      if constexpr (SEQ)
        if (later && tile >= part)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = 8 * (i / 4) + i % 4 < hidden - 32 * tile - 4 * h ? s[i] : 0.0f;
      Frag ds[D::FR];
#pragma unroll
      for (int f = 0; f < D::FR; ++f) ds[f] = Op<T>::from_acc(s, f);
#pragma unroll
      for (int d = 0; d < D::DT; ++d)
#pragma unroll
        for (int f = 0; f < D::FR; ++f) {
          dq[d] = Op<T>::mma(as_frag<Frag>(sh[buf][(2 * D::UNITS + d * D::FR + f) * 64 + lane]), ds[f], dq[d]);
          pace<T, DP>(f);
        }
    }
    if (BUFS == 1) {
      __syncthreads();
      if (t + 1 < it.b1) fetch(t + 1, 0);
    }
    wait_copies();
    __syncthreads();
  }
  if (active)
    finish_grad<T, DP>(a, it, tl, wave, lane, true, a.dq, a.ldq, a.part_q, a.q_quad, dq, a.scale);
}

// grad_k and grad_v: a wave keeps 32 keys and walks the query tiles (all heads
// of the group): S = Q K^T, P = exp2(S - lse), dV^T += dO^T P, dP = dO V^T,
// dS = P (dP - delta), dK^T += Q^T dS. PART 0: both (one_pass); else as PART 1
// (grad_v) and 2 (grad_k).
template <typename T, int DP, int PART, bool SEQ>
__device__ __forceinline__ void dkv_item(const BwdArgs& a, const Item& it, u32x4* pool, float* row_pool,
                                         int* hidden_pool) {
  using D = Dims<T, DP>;
  using Frag = typename Op<T>::Frag;
  constexpr bool WANT_V = PART != 2, WANT_K = PART != 1;
  constexpr int FORMS = dkv_forms(PART);
  constexpr int GC = 1, GR = WANT_V ? 2 : 1, QC = GR + 1;  // place of a form in the stage (Q rows: 0)
  constexpr int STAGE = FORMS * D::UNITS, PER = (STAGE + 3) / 4;
  constexpr int BUFS = stage_buffers(STAGE);
  const auto sh = reinterpret_cast<u32x4(*)[STAGE * 64]>(pool);
  const auto rows = reinterpret_cast<float(*)[64]>(row_pool);
  const auto hidden = reinterpret_cast<int(*)[32]>(hidden_pool);  // causal: of every query row of a tile
  const int lane = int(threadIdx.x) % 64, wave = wave_id(), n = lane % 32, h = lane / 32;
  const bool active = wave < it.tiles;
  const int kt = it.a0 + (active ? wave : 0);
  const Tile tl = ldc(a.ktiles + kt);
  const int64_t kat = (int64_t(kt) * a.groups + it.hk) * D::TILE;
  constexpr bool kReread = D::kShort && WANT_K;
  const T* const krows = a.kforms<T>(kKRows) + kat;
  Frag k[kReread ? 1 : D::KSTEPS], v[WANT_K ? D::KSTEPS : 1];
#pragma unroll
  for (int t = 0; t < D::KSTEPS; ++t) {
    if constexpr (!kReread) k[t] = as_frag<Frag>(unit16(krows, t, lane));
    if (WANT_K) v[t] = as_frag<Frag>(unit16(a.kforms<T>(kVRows) + kat, t, lane));
  }
  const float bias = a.bias[int64_t(kt) * 32 + n];
  // causal: keys that all samples share are seen by every query
  const bool later = SEQ && a.causal && kt >= a.shared;
  f32x16 dk[WANT_K ? D::DT : 1], dv[WANT_V ? D::DT : 1];
#pragma unroll
  for (int d = 0; d < D::DT; ++d) {
    if (WANT_K) dk[d] = zero16();
    if (WANT_V) dv[d] = zero16();
  }
  const auto fetch = [&](int tile, int buf) {
    const int64_t at = int64_t(tile) * a.groups + it.hk;
    const T* base = a.qforms<T>(0) + at * D::TILE;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = i * 4 + wave;
      if (u >= STAGE) break;
      // the forms in use, in their order in memory
      const int form = u / D::UNITS + (WANT_V || u < D::UNITS ? 0 : 1);
      copy_unit(base + form * a.qstride, u % D::UNITS, lane, &sh[buf][u * 64]);
    }
    if (threadIdx.x < 64) rows[buf][threadIdx.x] = a.rows[at * 64 + threadIdx.x];
    if constexpr (SEQ)
      if (a.causal && threadIdx.x < 32) {
        const Tile ql = ldc(a.qtiles + tile);
        hidden[buf][threadIdx.x] = hidden_from(a, ldc(a.reach + tile), ql.row0 + min(int(threadIdx.x), ql.n - 1));
      }
  };
  if (it.b0 < it.b1) fetch(it.b0, 0);
  wait_copies();
  __syncthreads();
  for (int t = it.b0; t < it.b1; ++t) {
    const int buf = BUFS == 2 ? (t - it.b0) & 1 : 0;
    if (BUFS == 2 && t + 1 < it.b1) fetch(t + 1, buf ^ 1);
    bool some = true, all = true;
    if constexpr (SEQ)
      if (later) {
        some = 32 * kt < __builtin_amdgcn_readfirstlane(hidden[buf][31]);
        all = 32 * kt + 31 < __builtin_amdgcn_readfirstlane(hidden[buf][0]);
      }
    if (active && some) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int u = 0; u < D::KSTEPS; ++u) {
        const Frag ku = kReread ? as_frag<Frag>(unit16(krows, u, lane)) : k[kReread ? 0 : u];
        s = Op<T>::mma(as_frag<Frag>(sh[buf][u * 64 + lane]), ku, s);
        if (WANT_K) dp = Op<T>::mma(as_frag<Frag>(sh[buf][(GR * D::UNITS + u) * 64 + lane]), v[u], dp);
        pace<T, DP>(u);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f32x4 l2 = *reinterpret_cast<const f32x4*>(&rows[buf][8 * b + 4 * h]);
        const f32x4 de = *reinterpret_cast<const f32x4*>(&rows[buf][32 + 8 * b + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[4 * b + i] = exp2_fast(fmaf(s[4 * b + i], a.scale2, bias) - l2[i]);
          if (WANT_K) dp[4 * b + i] = s[4 * b + i] * (dp[4 * b + i] - de[i]);
        }
      }
      if constexpr (SEQ)
        if (!all)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const bool seen = 32 * kt + n < hidden[buf][8 * (i / 4) + 4 * h + i % 4];
            s[i] = seen ? s[i] : 0.0f;
            if (WANT_K) dp[i] = seen ? dp[i] : 0.0f;
          }
      Frag p[D::FR], ds[D::FR];
#pragma unroll
      for (int f = 0; f < D::FR; ++f) {
        if (WANT_V) p[f] = Op<T>::from_acc(s, f);
        if (WANT_K) ds[f] = Op<T>::from_acc(dp, f);
      }
#pragma unroll
      for (int d = 0; d < D::DT; ++d)
#pragma unroll
        for (int f = 0; f < D::FR; ++f) {
          if (WANT_V)
            dv[d] = Op<T>::mma(as_frag<Frag>(sh[buf][(GC * D::UNITS + d * D::FR + f) * 64 + lane]), p[f], dv[d]);
          if (WANT_K)
            dk[d] = Op<T>::mma(as_frag<Frag>(sh[buf][(QC * D::UNITS + d * D::FR + f) * 64 + lane]), ds[f], dk[d]);
          pace<T, DP>(f);
        }
    }
    if (BUFS == 1) {
      __syncthreads();
      if (t + 1 < it.b1) fetch(t + 1, 0);
    }
    wait_copies();
    __syncthreads();
  }
  if (!active) return;
  // a masked key's gradients are 0 whatever the queries hold (its weights are, unless a
  // score or an lse is NaN)
  if (bias < 0.0f)
#pragma unroll
    for (int d = 0; d < D::DT; ++d) {
      if (WANT_K) dk[d] = zero16();
      if (WANT_V) dv[d] = zero16();
    }
  if constexpr (WANT_V)
    if (a.dv) finish_grad<T, DP>(a, it, tl, wave, lane, false, a.dv, a.ldk, a.part_v, a.k_quad, dv, 1.0f);
  if constexpr (WANT_K)
    if (a.dk) finish_grad<T, DP>(a, it, tl, wave, lane, false, a.dk, a.ldk, a.part_k, a.k_quad, dk, a.scale);
}

// All gradients in one launch: the items of the three kinds fill the device
// together and end together (a ragged batch's three launches each left a quarter
// of it idle at their end). Bound: matrix cores, exponentials and operand reads
// from shared memory (1 KB a product and wave) after one another: 448 us for a
// ragged bf16 batch of heads of 144, matrix cores busy 38 %; fp32, heads of 128, 165 us,
// 73 %. Workgroups of 8 waves copy half as much and were no faster (644 us against
// 641 us for the whole step), nor were wave priorities.
template <typename T, int DP>
constexpr int bwd_units() {
  constexpr int U = Dims<T, DP>::UNITS;
  // grad_q and grad_k: 3 forms; grad_v: 2, which may be kept twice where 3 are not
  constexpr int a = stage_units(3 * U), b = stage_units(dkv_forms(one_pass(DP, sizeof(T)) ? 0 : 1) * U);
  return a > b ? a : b;
}
template <typename T, int DP, bool SEQ>
__global__ __launch_bounds__(kThreads, lds_waves(bwd_units<T, DP>())) void bwd_kernel(BwdArgs a) {
  __shared__ u32x4 pool[bwd_units<T, DP>() * 64];
  __shared__ __attribute__((aligned(16))) float rows[2 * 64];
  __shared__ __attribute__((aligned(16))) int hidden[SEQ ? 2 * 32 : 4];
  const Item it = ldc(a.items + blockIdx.x);
  if (it.tiles == 0) return;
  if (it.kind == kItemQ) {
    if (a.dq) dq_item<T, DP, SEQ>(a, it, pool, rows);
  } else if constexpr (one_pass(DP, sizeof(T))) {
    if (a.dk || a.dv) dkv_item<T, DP, 0, SEQ>(a, it, pool, rows, hidden);
  } else if (it.kind == kItemV) {
    if (a.dv) dkv_item<T, DP, 1, SEQ>(a, it, pool, rows, hidden);
  } else {
    if (a.dk) dkv_item<T, DP, 2, SEQ>(a, it, pool, rows, hidden);
  }
}

// Columns 32 d .. of a wave's gradient: a part, or final rows (as finish_grad).
template <typename T, int DP>
__device__ __forceinline__ void put_columns(const BwdArgs& a, const Item& it, const Tile& tl, int within, bool query,
                                            int d, void* dst, int64_t ld, float* part, const f32x16& g, float scale) {
  const int n = lane_id() % 32, h = lane_id() / 32;
  if (it.slot >= 0) {
    store_columns(part + ((int64_t(it.slot) * it.stride + within) * 32 + n) * DP + 32 * d, h, g, scale);
  } else if (n < tl.n) {
    const int row = tl.row0 + n, G = query ? a.G : 1;
    scatter_columns(static_cast<T*>(dst) + int64_t(row / G) * ld, a.table, query, it.hk * G + row % G, h, d, g, scale);
  }
}
// s += A B^T of two packed tiles' rows.
template <typename T, int DP>
__device__ __forceinline__ void row_products(f32x16& s, const T* a, const T* b) {
  using Frag = typename Op<T>::Frag;
#pragma unroll 4
  for (int u = 0; u < Dims<T, DP>::KSTEPS; ++u)
    s = Op<T>::mma(as_frag<Frag>(unit16(a, u, lane_id())), as_frag<Frag>(unit16(b, u, lane_id())), s);
  __builtin_amdgcn_sched_barrier(0);
}

// Columns 32 d .. of grad_q of tile `within` of an item once more, as dq_item, of seen pairs alone.
template <typename T, int DP>
__device__ __forceinline__ void redo_dq(const BwdArgs& a, const Item& it, int within, int d) {
  using D = Dims<T, DP>;
  const int n = lane_id() % 32, h = lane_id() / 32;
  const Tile tl = ldc(a.qtiles + it.a0 + within);
  const Reach re = ldc(a.reach + it.a0 + within);
  const int64_t qat = int64_t(it.a0 + within) * a.groups + it.hk;
  const float lse2 = a.rows[qat * 64 + n], delta = a.rows[qat * 64 + 32 + n];
  // (where these are NaN, so is the row)
  if (!__any(n < tl.n && lse2 == lse2 && delta == delta)) return;
  const int hidden = hidden_from(a, re, tl.row0 + min(n, tl.n - 1));
  f32x16 dq = zero16();
#pragma unroll 1
  for (int t = it.b0; t < it.b1; ++t) {
    const int tile = key_tile<true>(a, re.skip, t);
    const int64_t kat = (int64_t(tile) * a.groups + it.hk) * D::TILE;
    f32x16 s = zero16(), dp = zero16();
    row_products<T, DP>(s, a.kforms<T>(kKRows) + kat, a.qforms<T>(kQRows) + qat * D::TILE);
    row_products<T, DP>(dp, a.kforms<T>(kVRows) + kat, a.qforms<T>(kGRows) + qat * D::TILE);
    SeenWeights<T> x;
    x.seen = t < a.shared ? 0xffffu : seen_below(32 * tile, hidden, h);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float bias = a.bias[int64_t(tile) * 32 + 8 * (i / 4) + 4 * h + i % 4];
      const float p = exp2_fast(fmaf(s[i], a.scale2, bias) - lse2);
      s[i] = x.seen >> i & 1 ? p * (dp[i] - delta) : 0.0f;
    }
#pragma unroll
    for (int f = 0; f < D::FR; ++f) x.w[f] = Op<T>::from_acc(s, f);
    __builtin_amdgcn_sched_barrier(0);
    add_seen(dq, a.kforms<T>(kKCols) + kat, d, x);
  }
  put_columns<T, DP>(a, it, tl, within, true, d, a.dq, a.ldq, a.part_q, dq, a.scale);
}

// Columns 32 d .. of grad_v, or of grad_k where `key`, as dkv_item.
template <typename T, int DP>
__device__ __forceinline__ void redo_dkv(const BwdArgs& a, const Item& it, int within, bool key, int d) {
  using D = Dims<T, DP>;
  const int n = lane_id() % 32, h = lane_id() / 32, kt = it.a0 + within;
  const Tile tl = ldc(a.ktiles + kt);
  const int64_t kat = (int64_t(kt) * a.groups + it.hk) * D::TILE;
  const float bias = a.bias[int64_t(kt) * 32 + n];
  f32x16 g = zero16();
#pragma unroll 1
  for (int t = it.b0; t < it.b1; ++t) {
    const int64_t at = int64_t(t) * a.groups + it.hk, qat = at * D::TILE;
    const Tile ql = ldc(a.qtiles + t);
    const Reach re = ldc(a.reach + t);
    f32x16 s = zero16(), dp = zero16();
    row_products<T, DP>(s, a.qforms<T>(kQRows) + qat, a.kforms<T>(kKRows) + kat);
    if (key) row_products<T, DP>(dp, a.qforms<T>(kGRows) + qat, a.kforms<T>(kVRows) + kat);
    SeenWeights<T> x;
    x.seen = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 8 * (i / 4) + 4 * h + i % 4;
      const bool seen = 32 * kt + n < hidden_from(a, re, ql.row0 + min(r, ql.n - 1));
      x.seen |= (seen ? 1u : 0u) << i;
      const float p = exp2_fast(fmaf(s[i], a.scale2, bias) - a.rows[at * 64 + r]);
      s[i] = !seen ? 0.0f : key ? p * (dp[i] - a.rows[at * 64 + 32 + r]) : p;
    }
#pragma unroll
    for (int f = 0; f < D::FR; ++f) x.w[f] = Op<T>::from_acc(s, f);
    __builtin_amdgcn_sched_barrier(0);
    add_seen(g, a.qforms<T>(key ? kQCols : kGCols) + qat, d, x);
  }
  if (bias < 0.0f) g = zero16();  // (as in dkv_item)
  put_columns<T, DP>(a, it, tl, within, false, d, key ? a.dk : a.dv, a.ldk, key ? a.part_k : a.part_v, g,
                     key ? a.scale : 1.0f);
}

// Causal batches: gradients of tiles that some keys or queries with infinities or NaN are
// hidden from in part, formed again after bwd_kernel wrote them. A wave looks at the flags of
// 2^shift tiles of the items, all at once, and the workgroup's waves take what has to be formed again, hardly
// ever any, in turn, 32 columns at a time: 4.6 us (ragged batch; one tile a wave, whatever their
// number, 13 us; a test for NaN at the end of bwd_kernel cost that 10 us of 340 by the registers). With NaN in all
// of grad_out a backward of 1500 rows, 4 heads of 128, takes 215 us for 66 in bf16 and 810 us for 168 in fp32.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads, 2) void redo_kernel(BwdArgs a, int items, int shift) {
  constexpr bool kBoth = one_pass(DP, sizeof(T));
  constexpr int DT = DP / 32;
  __shared__ uint32_t found[4];
  const int lane = lane_id(), wave = wave_id(), per = 1 << shift, lanes = 64 >> shift;
  const int first = int(blockIdx.x) * 4 * per, mine = first + wave * per + lane / lanes, sub = lane % lanes;
  const auto wants = [&](const Item& it, bool key) {
    return key ? a.dk && (kBoth || it.kind == kItemK) : a.dv && (kBoth || it.kind == kItemV);
  };
  // the first place hidden from a query tile's first row
  const auto hidden_first = [&](int tile) { return hidden_from(a, a.reach[tile], a.qtiles[tile].row0); };
  bool bad = false;
  if (mine < 4 * items) {
    const Item it = a.items[mine / 4];
    const int at = it.a0 + mine % 4;
    if (mine % 4 >= it.tiles) {
    } else if (it.kind == kItemQ) {
      if (a.dq) {
        const int part = hidden_first(at) >> 5, skip = a.reach[at].skip;
        for (int t = it.b1 - 1 - sub; t >= max(it.b0, a.shared) && !bad; t -= lanes) {
          const int tile = key_tile<true>(a, skip, t);
          if (tile < part) break;
          bad = a.k_bad[int64_t(tile) * a.groups + it.hk] != 0;
        }
      }
    } else if (at >= a.shared && (wants(it, false) || wants(it, true))) {
      for (int t = it.b0 + sub; t < it.b1 && !bad; t += lanes) {
        if (32 * at + 31 < hidden_first(t)) break;
        bad = a.q_bad[int64_t(t) * a.groups + it.hk] != 0;
      }
    }
  }
  const uint64_t which_bad = __ballot(bad);
  uint32_t some = 0;
  for (int e = 0; e < per; ++e) some |= (which_bad >> (lanes * e) & (~uint64_t(0) >> (64 - lanes)) ? 1u : 0u) << e;
  if (lane == 0) found[wave] = some;
  __syncthreads();
  int turn = 0;
  for (uint32_t left = found[0] | found[1] << per | found[2] << 2 * per | found[3] << 3 * per; left; left &= left - 1) {
    const int which = first + __builtin_amdgcn_readfirstlane(__builtin_ctz(left)), w = which % 4;
    const Item it = ldc(a.items + which / 4);
    if (it.kind == kItemQ) {
#pragma unroll 1
      for (int d = 0; d < DT; ++d)
        if (turn++ % 4 == wave) redo_dq<T, DP>(a, it, w, d);
      continue;
    }
    // (a query whose lse is NaN makes NaN of all keys that it sees: nothing to mend where all see one)
    bool nan = false;
    for (int t = it.b1 - 1; t >= it.b0 && 32 * (it.a0 + w) + 31 < hidden_first(t) && !nan; --t) {
      const float lse2 = a.rows[(int64_t(t) * a.groups + it.hk) * 64 + lane % 32];
      nan = __any(lse2 != lse2);
    }
    if (nan) continue;
#pragma unroll 1
    for (int d = 0; d < 2 * DT; ++d)
      if (wants(it, d >= DT) && turn++ % 4 == wave) redo_dkv<T, DP>(a, it, w, d >= DT, d % DT);
  }
}

// Adds the parts of split gradient rows in order, as fwd_join_kernel.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void grad_join_kernel(GradJoinArgs a) {
  const Join j = ldc(a.joins + blockIdx.x);
  const Tile tl = ldc(a.tiles + j.tile);
  const int n = int(threadIdx.x) / 8, d = int(blockIdx.y) * 32 + int(threadIdx.x) % 8 * 4;
  if (n >= tl.n) return;
  const float* p = (blockIdx.z ? a.part1 : a.part0) + ((int64_t(j.slot) * j.stride + j.within) * 32 + n) * DP + d;
  float v[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int k = 0; k < j.parts; ++k) {
    const f32x4 o = *reinterpret_cast<const f32x4*>(p + int64_t(k) * j.stride * 32 * DP);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += o[i];
  }
  const int row = tl.row0 + n, token = row / a.G, head = j.hk * a.G + row % a.G;
  scatter4(static_cast<T*>(blockIdx.z ? a.dst1 : a.dst0) + int64_t(token) * a.ld, a.table, d, a.query, head, a.quad, v);
}

// -------------------------------------------------------------------- launch

template <typename T, int DP>
struct Kernels {
  static void pack(const PackArgs& a, hipStream_t s) {
    const bool grads = a.rows_out != nullptr, vec = a.t[0].vec && a.t[1].vec && (!grads || a.out_vec);
    const auto k = vec ? (grads ? pack_kernel<T, DP, true, true> : pack_kernel<T, DP, true, false>)
                       : (grads ? pack_kernel<T, DP, false, true> : pack_kernel<T, DP, false, false>);
    hipLaunchKernelGGL(k, dim3(unsigned((a.ntiles + 7) / 8 * 8 * a.groups)), dim3(kThreads), 0, s, a);
  }
  static void fwd(const FwdArgs& a, int items, int tiles, hipStream_t s) {
    if (tiles == 1) hipLaunchKernelGGL((fwd_few_kernel<T, DP, false>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
    if (tiles == 4) hipLaunchKernelGGL((fwd_kernel<T, DP, 1, false>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
    if constexpr (wide_forward(DP, sizeof(T)))
      if (tiles == 8) hipLaunchKernelGGL((fwd_kernel<T, DP, 2, false>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
  }
  static void fwd_join(const FwdArgs& a, int joins, hipStream_t s) {
    hipLaunchKernelGGL((fwd_join_kernel<T, DP>), dim3(unsigned(joins), DP / 32), dim3(kThreads), 0, s, a);
  }
  static void bwd(const BwdArgs& a, int items, hipStream_t s) {
    hipLaunchKernelGGL((bwd_kernel<T, DP, false>), dim3(unsigned(items)), dim3(kThreads), 0, s, a);
  }
  static void grad_join(const GradJoinArgs& a, int joins, int tensors, hipStream_t s) {
    hipLaunchKernelGGL((grad_join_kernel<T, DP>), dim3(unsigned(joins), DP / 32, unsigned(tensors)), dim3(kThreads), 0,
                       s, a);
  }
  static KernelTable table() { return {pack, fwd, fwd_join, bwd, grad_join}; }
};

}  // namespace attn
}  // namespace cgtp
