// Group norm of irreps rows with the activation of the even scalars, channels
// last, over ragged samples.
//
// Per sample and group: mu = mean x for 0e blocks (else 0), var = mean (x-mu)^2
// over the sample's rows, the 2l+1 components and the group's channels,
// xh = (x - mu) / sqrt(var + eps), z = xh w_c (+ b_c), y = act(z). Backward, with
// gz = g act'(z), A_c = sum gz xh, B_c = sum gz per sample and channel:
//   gx = r (gz w_c - [0e] sum_c w_c B_c / n - xh sum_c w_c A_c / n)
// so one set of per-channel sums gives both the weights' gradients and the two
// means that grad_x needs.
//
// Bound: memory. A workgroup takes one run of a sample's rows (RowChunk) and one
// strip of a block (whole groups, NormStrip); lanes lie along the channels (16
// bytes each), so a wave reads whole runs of a component. Statistics: every
// thread sums x - p and (x - p)^2 about its own first value p, which keeps the
// sums free of cancellation, and means and squares are merged pairwise in a
// fixed tree. All sums are in fp32 (fp64 for fp64 storage).
//
// Measured, fp32, 24,000 rows of 1152: statistics 19 us (5.9 TB/s), y 45 us (4.9),
// backward's sums 35 us (6.4), grad_x 51 us (6.5); bf16, 96 samples of 20 - 220 rows in
// one launch forward and two backward: 20 us and 31 + 4 us.
#include <algorithm>
#include <type_traits>

#include "device_util.hpp"
#include "layers.hpp"

namespace cgtp {

namespace {

constexpr int kNT = 256;        // threads of a run's workgroup
constexpr int kNTS = 256;      // of a whole sample's

// Which unit (run or sample) and strip a workgroup takes. Strips fastest: the
// strips of a run read the same rows, i.e. the same memory pages, together (fp32
// box of 24000 rows: 155 us against 165 us); units fastest: the strips with the
// most work come first, which matters when the launch is more than the device
// holds at once (the 104,217 rows above: 270 us against 330 us).
struct Order {
  int units, strips;
  bool strips_fastest;
  __device__ __forceinline__ int unit() const {
    return strips_fastest ? int(blockIdx.x) / strips : int(blockIdx.x) % units;
  }
  __device__ __forceinline__ int strip() const {
    return strips_fastest ? int(blockIdx.x) % strips : int(blockIdx.x) / units;
  }
};

template <typename A>
__device__ __forceinline__ A rsqrt_acc(A v);
template <>
__device__ __forceinline__ float rsqrt_acc(float v) { return rsqrtf(v); }
template <>
__device__ __forceinline__ double rsqrt_acc(double v) { return 1.0 / sqrt(v); }

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }
__device__ __forceinline__ double sigmoid(double z) { return 1.0 / (1.0 + exp(-z)); }
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.70710678118654752f * z); }
__device__ __forceinline__ double normal_cdf(double z) { return 0.5 * erfc(-0.70710678118654752 * z); }
__device__ __forceinline__ float normal_pdf(float z) { return 0.39894228040143268f * __expf(-0.5f * z * z); }
__device__ __forceinline__ double normal_pdf(double z) { return 0.39894228040143268 * exp(-0.5 * z * z); }

template <typename A>
__device__ __forceinline__ A act_value(int act, A z) {
  if (act == CGTP_ACT_SILU) return z * sigmoid(z);
  if (act == CGTP_ACT_GELU) return z * normal_cdf(z);
  return z;
}
template <typename A>
__device__ __forceinline__ A act_slope(int act, A z) {
  if (act == CGTP_ACT_SILU) {
    const A s = sigmoid(z);
    return s * (A(1) + z * (A(1) - s));
  }
  if (act == CGTP_ACT_GELU) return normal_cdf(z) + z * normal_pdf(z);
  return A(1);
}

// Where a thread works: lane `lane` of `per` along the strip's channels (VEC
// each; a group wider than 256 lanes is walked in steps), every slots-th row
// from slot on.
struct Place {
  int per, slots, slot, lane, lanes, chan0;
};
template <int VEC, int NT>
__device__ __forceinline__ Place place(const NormStrip& st) {
  Place p;
  p.lanes = st.ng * st.cg / VEC;
  p.per = p.lanes < NT ? p.lanes : NT;
  p.slots = NT / p.per;
  p.slot = int(threadIdx.x) / p.per;
  p.lane = int(threadIdx.x) % p.per;
  p.chan0 = st.g0 * st.cg;
  return p;
}

template <typename A>
struct Moments {
  A n, mean, m2;
};
template <typename A>
struct alignas(4 * sizeof(A)) Part {
  A n, mean, m2, pad;
};
template <typename A>
__device__ __forceinline__ Moments<A> merge(const Moments<A>& a, const Moments<A>& b) {
  const A n = a.n + b.n;
  if (!(n > A(0))) return a;
  const A d = b.mean - a.mean, f = b.n / n;
  return {n, a.mean + d * f, a.m2 + b.m2 + d * d * a.n * f};
}

// VEC elements as stored: what a load in flight occupies.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Raw {
  T e[VEC];
};

// Rows kept in flight by a thread: about 8 accesses of one or two tensors.
template <int NC, int TENSORS>
struct RowsAhead {
  static constexpr int value = TENSORS == 1 ? (NC == 1 ? 4 : NC <= 5 ? 2 : 1) : (NC == 1 ? 4 : NC == 3 ? 2 : 1);
};

// Every slots-th of the n rows from the thread's slot on: f(first, count) with
// `count` (an integral constant) rows first, first + slots, ... Whole batches
// first, so that no load in them stands under a condition (where it would wait
// for its use), then single rows.
template <int RU, typename F>
__device__ __forceinline__ void walk(const Place& p, int n, F&& f) {
  int r = p.slot;
  if constexpr (RU > 1)
    for (; r + (RU - 1) * p.slots < n; r += RU * p.slots) f(r, std::integral_constant<int, RU>{});
  for (; r < n; r += p.slots) f(r, std::integral_constant<int, 1>{});
}

// NC components of `count` rows from row r on; base is the same for the whole
// workgroup, the lane's part of the address fits 32 bits (rows of at most 2^18
// elements, runs of them cut at 2^12 rows).
template <typename T, int VEC, int NC, int RU>
__device__ __forceinline__ void load_rows(const T* base, const Place& p, int lane_off, int dim, int mul, int r,
                                          Raw<T, VEC> (&v)[RU][NC]) {
#pragma unroll
  for (int u = 0; u < RU; ++u)
#pragma unroll
    for (int m = 0; m < NC; ++m)
      v[u][m] = *reinterpret_cast<const Raw<T, VEC>*>(base + m * mul + uint32_t((r + u * p.slots) * dim + lane_off));
}

// Results are not read again soon: stored past the caches, they leave the rows
// there for the second pass (and leave no dirty lines for later calls to wait for:
// on 104,217 rows of 4 KB the first pass took 95 us instead of 128).
template <typename R>
__device__ __forceinline__ void put(R* p, const R& v) {
  if constexpr (sizeof(R) == 16) {
    typedef uint32_t V __attribute__((ext_vector_type(4)));
    V t;
    __builtin_memcpy(&t, &v, 16);
    __builtin_nontemporal_store(t, reinterpret_cast<V*>(p));
  } else {
    *p = v;
  }
}

// f(base row, rows) over at most 2^12 rows at a time.
template <typename F>
__device__ __forceinline__ void spans(int r0, int r1, F&& f) {
  for (int r = r0; r < r1; r += 4096) f(r, min(4096, r1 - r));
}

// Moments of the thread's elements of channel vector `lane0`. Only the even
// scalars take a mean.
template <typename T, int VEC, int NC, typename A = typename AccOf<T>::type>
__device__ __forceinline__ Moments<A> thread_moments(const NormStrip& st, const Place& p, int lane0, int r0, int r1,
                                                     const T* x, int64_t dim) {
  const bool even = NC == 1 && st.bias >= 0;
  const int lane_off = lane0 * VEC;
  A s1 = 0, s2 = 0, pivot = 0;
  int n = 0;
  if (even && r0 + p.slot < r1) pivot = to_acc<A>(x[int64_t(r0 + p.slot) * dim + st.off + p.chan0 + lane_off]);
  spans(r0, r1, [&](int rs, int rows) {
    const T* base = x + int64_t(rs) * dim + st.off + p.chan0;
    walk<RowsAhead<NC, 1>::value>(p, rows, [&](int r, auto count) {
      constexpr int RU = decltype(count)::value;
      Raw<T, VEC> v[RU][NC];
      load_rows<T, VEC, NC, RU>(base, p, lane_off, int(dim), st.mul, r, v);
      n += RU;
#pragma unroll
      for (int u = 0; u < RU; ++u)
#pragma unroll
        for (int m = 0; m < NC; ++m)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            A d = to_acc<A>(v[u][m].e[i]);
            if (NC == 1) {
              d -= pivot;
              s1 += d;
            }
            s2 += d * d;
          }
    });
  });
  if (n == 0) return {A(0), A(0), A(0)};
  const A count = A(n) * A(VEC * NC);
  if (!even) return {count, A(0), s2};
  const A f = s1 / count;
  const A m2 = s2 - s1 * f;
  return {count, pivot + f, m2 > A(0) || m2 != m2 ? m2 : A(0)};
}

// Fixed tree over the threads of each group; the result of group g is left in
// sh[g * (lanes per group)].
template <typename A>
__device__ __forceinline__ void group_tree(Moments<A>* sh, const Place& p, int lanes_per_group) {
  __syncthreads();
  for (int cur = p.slots; cur > 1;) {
    const int half = (cur + 1) / 2;
    if (p.slot + half < cur) sh[threadIdx.x] = merge(sh[threadIdx.x], sh[threadIdx.x + half * p.per]);
    cur = half;
    __syncthreads();
  }
  const int in_group = p.lane % lanes_per_group;
  for (int cur = lanes_per_group; cur > 1;) {
    const int half = (cur + 1) / 2;
    if (p.slot == 0 && in_group + half < cur) sh[threadIdx.x] = merge(sh[threadIdx.x], sh[threadIdx.x + half]);
    cur = half;
    __syncthreads();
  }
}

template <int VEC, int NT>
__device__ __forceinline__ int lanes_of_group(const NormStrip& st, const Place& p) {
  return p.lanes > NT ? NT : st.cg / VEC;
}

// Moments of the groups of one strip over rows r0 .. r1, left in sh.
template <int NT, typename T, int VEC, int NC, typename A>
__device__ __forceinline__ void strip_moments(const NormStrip& st, const Place& p, int r0, int r1, const T* x,
                                              int64_t dim, Moments<A>* sh) {
  Moments<A> t{A(0), A(0), A(0)};
  if (p.slot < p.slots)
    for (int l = p.lane; l < p.lanes; l += NT) t = merge(t, thread_moments<T, VEC, NC>(st, p, l, r0, r1, x, dim));
  sh[threadIdx.x] = t;
  group_tree(sh, p, lanes_of_group<VEC, NT>(st, p));
}

#define CGTP_NC_SWITCH(nc, CALL) \
  switch (nc) {                  \
    case 1: CALL(1); break;      \
    case 3: CALL(3); break;      \
    case 5: CALL(5); break;      \
    case 7: CALL(7); break;      \
    default: CALL(9); break;     \
  }

// Count, mean and centred square sum of every group over one run of rows:
// part [chunk][groups].
template <typename T, int VEC>
__global__ __launch_bounds__(kNT) void norm_moments_kernel(const RowChunk* chunks, const NormStrip* strips, const T* x,
                                                           int64_t dim, int num_groups, int chunk_first, Order ord,
                                                           Part<typename AccOf<T>::type>* part) {
  using A = typename AccOf<T>::type;
  __shared__ Moments<A> sh[kNT];
  const int chunk = chunk_first + ord.unit();
  const RowChunk ch = ldc(chunks + chunk);
  const NormStrip st = ldc(strips + ord.strip());
  const Place p = place<VEC, kNT>(st);
#define CALL(N) strip_moments<kNT, T, VEC, N, A>(st, p, ch.r0, ch.r1, x, dim, sh)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
  const int lg = lanes_of_group<VEC, kNT>(st, p);
  if (int(threadIdx.x) < st.ng) {
    const Moments<A> g = sh[threadIdx.x * lg];
    part[int64_t(chunk) * num_groups + st.gid + threadIdx.x] = {g.n, g.mean, g.m2, A(0)};
  }
}

// y of the thread's channels over rows r0 .. r1 from the group's mean and rstd.
template <int NT, typename T, int VEC, int NC, typename A>
__device__ __forceinline__ void strip_apply(const NormStrip& st, const Place& p, int r0, int r1, const T* x, T* y,
                                            int64_t dim, const T* w, const T* b, const A* mean, const A* rstd,
                                            int act) {
  if (p.slot >= p.slots) return;
  for (int l = p.lane; l < p.lanes; l += NT) {
    const int c0 = p.chan0 + l * VEC, g = l * VEC / st.cg;
    const A mu = mean[g], rs = rstd[g];
    A a[VEC], sft[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      a[i] = w ? rs * to_acc<A>(w[st.chan + c0 + i]) : rs;
      sft[i] = NC == 1 && st.bias >= 0 && b ? to_acc<A>(b[st.bias + c0 + i]) : A(0);
    }
    const int on = NC == 1 && st.bias >= 0 ? act : int(CGTP_ACT_NONE);
    spans(r0, r1, [&](int first, int rows) {
      const int64_t at = int64_t(first) * dim + st.off + p.chan0;
      walk<RowsAhead<NC, 1>::value>(p, rows, [&](int r, auto count) {
        constexpr int RU = decltype(count)::value;
        Raw<T, VEC> v[RU][NC];
        load_rows<T, VEC, NC, RU>(x + at, p, l * VEC, int(dim), st.mul, r, v);
#pragma unroll
        for (int u = 0; u < RU; ++u)
#pragma unroll
          for (int m = 0; m < NC; ++m) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const A e = to_acc<A>(v[u][m].e[i]);
              from_acc(v[u][m].e[i], NC == 1 ? act_value(on, (e - mu) * a[i] + sft[i]) : e * a[i]);
            }
            put(reinterpret_cast<Raw<T, VEC>*>(y + at + m * st.mul + uint32_t((r + u * p.slots) * int(dim) + l * VEC)),
                v[u][m]);
          }
      });
    });
  }
}

// The strip's means and reciprocal deviations from its groups' moments (thread g
// holds group g), kept in shared memory and, where wanted, in stats.
template <typename A>
__device__ __forceinline__ void publish(const NormStrip& st, const Moments<A>& g, A eps, A* mean, A* rstd, A* stats) {
  const A r = rsqrt_acc(g.m2 / g.n + eps);
  mean[threadIdx.x] = g.mean;
  rstd[threadIdx.x] = r;
  if (stats) {
    stats[2 * (st.gid + threadIdx.x)] = g.mean;
    stats[2 * (st.gid + threadIdx.x) + 1] = r;
  }
}

// Joins the runs' moments of a sample's groups and writes y of one run.
template <typename T, int VEC>
__global__ __launch_bounds__(kNT) void norm_apply_kernel(const RowChunk* chunks, const NormStrip* strips, const T* x,
                                                         T* y, int64_t dim, int num_groups, int chunk_first, Order ord,
                                                         const T* w, const T* b,
                                                         const Part<typename AccOf<T>::type>* part,
                                                         typename AccOf<T>::type* stats,
                                                         typename AccOf<T>::type eps, int act) {
  using A = typename AccOf<T>::type;
  __shared__ Moments<A> sh[kNT];
  __shared__ A mean[kNT], rstd[kNT];
  const RowChunk ch = ldc(chunks + chunk_first + ord.unit());
  const NormStrip st = ldc(strips + ord.strip());
  const Place p = place<VEC, kNT>(st);
  // kNT / ng threads a group, each a fixed part of the runs
  Place q;
  q.per = st.ng;
  q.slots = kNT / st.ng;
  q.slot = int(threadIdx.x) / st.ng;
  q.lane = int(threadIdx.x) % st.ng;
  q.lanes = q.chan0 = 0;
  Moments<A> t{A(0), A(0), A(0)};
  if (q.slot < q.slots)
#pragma unroll 4
    for (int k = q.slot; k < ch.nchunk; k += q.slots) {
      const Part<A> m = part[int64_t(ch.chunk0 + k) * num_groups + st.gid + q.lane];
      t = merge(t, Moments<A>{m.n, m.mean, m.m2});
    }
  sh[threadIdx.x] = t;
  group_tree(sh, q, 1);
  if (int(threadIdx.x) < st.ng)
    publish(st, sh[threadIdx.x], eps, mean, rstd,
            stats && ch.r0 == ch.row0 ? stats + int64_t(ch.sample) * num_groups * 2 : nullptr);
  __syncthreads();
#define CALL(N) strip_apply<kNT, T, VEC, N, A>(st, p, ch.r0, ch.r1, x, y, dim, w, b, mean, rstd, act)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
}

// A whole sample's strip by one workgroup, where samples are short: statistics,
// then y; the second read of x comes from the caches.
template <typename T, int VEC>
__global__ __launch_bounds__(kNTS) void norm_sample_kernel(const int32_t* first_row, const NormStrip* strips,
                                                          int sample_first, Order ord, const T* x, T* y, int64_t dim,
                                                          int num_groups, const T* w, const T* b,
                                                          typename AccOf<T>::type* stats,
                                                          typename AccOf<T>::type eps, int act) {
  using A = typename AccOf<T>::type;
  __shared__ Moments<A> sh[kNTS];
  __shared__ A mean[kNTS], rstd[kNTS];
  const int s = sample_first + ord.unit(), r0 = first_row[s], r1 = first_row[s + 1];
  if (r0 == r1) return;
  const NormStrip st = ldc(strips + ord.strip());
  const Place p = place<VEC, kNTS>(st);
#define CALL(N) strip_moments<kNTS, T, VEC, N, A>(st, p, r0, r1, x, dim, sh)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
  const int lg = lanes_of_group<VEC, kNTS>(st, p);
  if (int(threadIdx.x) < st.ng)
    publish(st, sh[threadIdx.x * lg], eps, mean, rstd, stats ? stats + int64_t(s) * num_groups * 2 : nullptr);
  __syncthreads();
#define CALL(N) strip_apply<kNTS, T, VEC, N, A>(st, p, r0, r1, x, y, dim, w, b, mean, rstd, act)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
}

// A_c and B_c of one run of rows: part [chunk][2][channels] (B_c only for even
// scalars, else 0).
template <int NT, typename T, int VEC, int NC, typename A>
__device__ __forceinline__ void strip_sums(const NormStrip& st, const Place& p, int r0, int r1, const T* x,
                                           const T* g, int64_t dim, const T* w, const T* b, const A* stats, int act,
                                           A* part, int channels, A (*sh)[2 * VEC + 1]) {
  constexpr int SUMS = NC == 1 ? 2 * VEC : VEC;
  for (int l0 = 0; l0 < p.lanes; l0 += NT) {
    const int l = l0 + p.lane, c0 = p.chan0 + l * VEC;
    A sum[SUMS];  // A_c, then B_c
#pragma unroll
    for (int i = 0; i < SUMS; ++i) sum[i] = A(0);
    if (p.slot < p.slots && l < p.lanes) {
      const int gi = l * VEC / st.cg;
      const A mu = stats[2 * gi], rs = stats[2 * gi + 1];
      A wv[NC == 1 ? VEC : 1], bv[NC == 1 ? VEC : 1];
      if constexpr (NC == 1)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          wv[i] = w ? to_acc<A>(w[st.chan + c0 + i]) : A(1);
          bv[i] = st.bias >= 0 && b ? to_acc<A>(b[st.bias + c0 + i]) : A(0);
        }
      const int on = NC == 1 && st.bias >= 0 ? act : int(CGTP_ACT_NONE);
      spans(r0, r1, [&](int first, int rows) {
        const int64_t at = int64_t(first) * dim + st.off + p.chan0;
        walk<RowsAhead<NC, 2>::value>(p, rows, [&](int r, auto count) {
          constexpr int RU = decltype(count)::value;
          Raw<T, VEC> v[RU][NC], d[RU][NC];
          load_rows<T, VEC, NC, RU>(x + at, p, l * VEC, int(dim), st.mul, r, v);
          load_rows<T, VEC, NC, RU>(g + at, p, l * VEC, int(dim), st.mul, r, d);
#pragma unroll
          for (int u = 0; u < RU; ++u)
#pragma unroll
            for (int m = 0; m < NC; ++m)
#pragma unroll
              for (int i = 0; i < VEC; ++i) {
                const A e = to_acc<A>(v[u][m].e[i]), gy = to_acc<A>(d[u][m].e[i]);
                if constexpr (NC == 1) {
                  const A xh = (e - mu) * rs, gz = gy * act_slope(on, xh * wv[i] + bv[i]);
                  sum[i] += gz * xh;
                  sum[VEC + i] += gz;
                } else {
                  sum[i] += gy * e;
                }
              }
        });
      });
      // (not of an empty sample, whose statistics are not written: 0 times them may be NaN)
      if (NC > 1 && r0 < r1)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] *= rs;
    }
#pragma unroll
    for (int i = 0; i < SUMS; ++i) sh[threadIdx.x][i] = sum[i];
    __syncthreads();
    for (int cur = p.slots; cur > 1;) {
      const int half = (cur + 1) / 2;
      if (p.slot + half < cur)
#pragma unroll
        for (int i = 0; i < SUMS; ++i) {
          sum[i] += sh[threadIdx.x + half * p.per][i];
          sh[threadIdx.x][i] = sum[i];
        }
      cur = half;
      __syncthreads();
    }
    if (p.slot == 0 && l < p.lanes)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        part[st.chan + c0 + i] = sum[i];
        part[channels + st.chan + c0 + i] = NC == 1 ? sum[SUMS - VEC + i] : A(0);
      }
    __syncthreads();
  }
}

template <typename T, int VEC>
__global__ __launch_bounds__(kNT) void norm_sums_kernel(const RowChunk* chunks, const NormStrip* strips, const T* x,
                                                        const T* g, int64_t dim, int num_groups, int channels,
                                                        int chunk_first, Order ord, const T* w, const T* b,
                                                        const typename AccOf<T>::type* stats, int act,
                                                        typename AccOf<T>::type* part) {
  using A = typename AccOf<T>::type;
  __shared__ A sh[kNT][2 * VEC + 1];
  const int chunk = chunk_first + ord.unit();
  const RowChunk ch = ldc(chunks + chunk);
  const NormStrip st = ldc(strips + ord.strip());
  const Place p = place<VEC, kNT>(st);
  const A* ss = stats + (int64_t(ch.sample) * num_groups + st.gid) * 2;
  A* o = part + int64_t(chunk) * 2 * channels;
#define CALL(N) strip_sums<kNT, T, VEC, N, A>(st, p, ch.r0, ch.r1, x, g, dim, w, b, ss, act, o, channels, sh)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
}

// Sums rows first[s] .. first[s + 1] of part [chunk][cols] into out [s][cols]:
// 8 columns and 32 rows at a time, fixed order.
template <typename A>
__global__ __launch_bounds__(kNT) void norm_join_kernel(const int32_t* first, int sample_first, const A* part, A* out,
                                                        int cols) {
  __shared__ A sh[32][9];
  const int s = sample_first + int(blockIdx.x), t = int(threadIdx.x) % 8, j = int(threadIdx.x) / 8;
  const int c = int(blockIdx.y) * 8 + t, end = first[s + 1];
  A v = 0;
  if (c < cols)
#pragma unroll 4
    for (int k = first[s] + j; k < end; k += 32) v += part[int64_t(k) * cols + c];
  sh[j][t] = v;
  __syncthreads();
  if (j == 0 && c < cols) {
    for (int k = 1; k < 32; ++k) v += sh[k][t];
    out[int64_t(s) * cols + c] = v;
  }
}

// grad_weight and grad_bias: the samples' sums [S][2][channels] added over S.
template <typename T>
__global__ __launch_bounds__(kNT) void norm_param_kernel(const NormStrip* strips, const typename AccOf<T>::type* sums,
                                                         int64_t S, int channels, T* gw, T* gb) {
  using A = typename AccOf<T>::type;
  __shared__ A sh[16][33];
  const NormStrip st = ldc(strips + blockIdx.y);
  const int j = int(threadIdx.x) / 16, t = int(threadIdx.x) % 16;
  for (int c0 = int(blockIdx.x) * 16; c0 < st.ng * st.cg; c0 += int(gridDim.x) * 16) {
    const int c = st.g0 * st.cg + c0 + t;
    const bool in = c0 + t < st.ng * st.cg;
    A a = 0, b = 0;
    if (in)
#pragma unroll 4
      for (int64_t s = j; s < S; s += 16) {
        const A* q = sums + s * 2 * channels + st.chan + c;
        a += q[0];
        b += q[channels];
      }
    sh[j][t] = a;
    sh[j][16 + t] = b;
    __syncthreads();
    if (j == 0 && in) {
      for (int k = 1; k < 16; ++k) {
        a += sh[k][t];
        b += sh[k][16 + t];
      }
      if (gw) from_acc(gw[st.chan + c], a);
      if (gb && st.bias >= 0) from_acc(gb[st.bias + c], b);
    }
    __syncthreads();
  }
}

// grad_x of one run of rows from its sample's per-channel sums.
template <int NT, typename T, int VEC, int NC, typename A>
__device__ __forceinline__ void strip_grad(const NormStrip& st, const Place& p, int r0, int r1, const T* x, const T* g,
                                           T* gx, int64_t dim, const T* w, const T* b, const A* stats, const A* mean_a,
                                           const A* mean_b, int act) {
  if (p.slot >= p.slots) return;
  for (int l = p.lane; l < p.lanes; l += NT) {
    const int c0 = p.chan0 + l * VEC, gi = l * VEC / st.cg;
    const A mu = stats[2 * gi], rs = stats[2 * gi + 1], ma = mean_a[gi], mb = mean_b[gi];
    A wv[VEC], bv[NC == 1 ? VEC : 1];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      wv[i] = w ? to_acc<A>(w[st.chan + c0 + i]) : A(1);
      if constexpr (NC == 1) bv[i] = st.bias >= 0 && b ? to_acc<A>(b[st.bias + c0 + i]) : A(0);
      else wv[i] *= rs;
    }
    const A ca = rs * rs * ma;
    const int on = NC == 1 && st.bias >= 0 ? act : int(CGTP_ACT_NONE);
    spans(r0, r1, [&](int first, int rows) {
      const int64_t at = int64_t(first) * dim + st.off + p.chan0;
      walk<RowsAhead<NC, 2>::value>(p, rows, [&](int r, auto count) {
        constexpr int RU = decltype(count)::value;
        Raw<T, VEC> v[RU][NC], d[RU][NC];
        load_rows<T, VEC, NC, RU>(x + at, p, l * VEC, int(dim), st.mul, r, v);
        load_rows<T, VEC, NC, RU>(g + at, p, l * VEC, int(dim), st.mul, r, d);
#pragma unroll
        for (int u = 0; u < RU; ++u)
#pragma unroll
          for (int m = 0; m < NC; ++m) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const A e = to_acc<A>(v[u][m].e[i]), gy = to_acc<A>(d[u][m].e[i]);
              if constexpr (NC == 1) {
                const A xh = (e - mu) * rs, gz = gy * act_slope(on, xh * wv[i] + bv[i]);
                from_acc(v[u][m].e[i], rs * (gz * wv[i] - mb - xh * ma));
              } else {
                from_acc(v[u][m].e[i], gy * wv[i] - e * ca);
              }
            }
            put(reinterpret_cast<Raw<T, VEC>*>(gx + at + m * st.mul + uint32_t((r + u * p.slots) * int(dim) + l * VEC)),
                v[u][m]);
          }
      });
    });
  }
}

// Means of w A and w B over the groups of a strip, from per-channel sums.
template <int NT, typename T, typename A>
__device__ __forceinline__ void group_means(const NormStrip& st, A count, const T* w, const A* sums, int channels,
                                            A* mean_a, A* mean_b, A* sha, A* shb) {
  // NT / ng threads a group (ng <= NT); fixed order
  const int slots = NT / st.ng, slot = int(threadIdx.x) / st.ng, gi = int(threadIdx.x) % st.ng;
  A a = 0, b = 0;
  if (slot < slots)
    for (int c = slot; c < st.cg; c += slots) {
      const int ch = st.chan + (st.g0 + gi) * st.cg + c;
      const A wc = w ? to_acc<A>(w[ch]) : A(1);
      a += wc * sums[ch];
      b += wc * sums[channels + ch];
    }
  sha[threadIdx.x] = a;
  shb[threadIdx.x] = b;
  __syncthreads();
  for (int cur = slots; cur > 1;) {
    const int half = (cur + 1) / 2;
    if (slot + half < cur) {
      sha[threadIdx.x] += sha[threadIdx.x + half * st.ng];
      shb[threadIdx.x] += shb[threadIdx.x + half * st.ng];
    }
    cur = half;
    __syncthreads();
  }
  if (int(threadIdx.x) < st.ng) {
    mean_a[threadIdx.x] = sha[threadIdx.x] / count;
    mean_b[threadIdx.x] = st.bias >= 0 ? shb[threadIdx.x] / count : A(0);
  }
  __syncthreads();
}

template <typename T, int VEC>
__global__ __launch_bounds__(kNT) void norm_grad_kernel(const RowChunk* chunks, const NormStrip* strips, const T* x,
                                                        const T* g, T* gx, int64_t dim, int num_groups, int channels,
                                                        int chunk_first, Order ord, const T* w, const T* b,
                                                        const typename AccOf<T>::type* stats,
                                                        const typename AccOf<T>::type* sums, int act) {
  using A = typename AccOf<T>::type;
  __shared__ A sha[kNT], shb[kNT], ma[kNT], mb[kNT];
  const RowChunk ch = ldc(chunks + chunk_first + ord.unit());
  const NormStrip st = ldc(strips + ord.strip());
  const Place p = place<VEC, kNT>(st);
  const A count = A(ch.rows) * A(st.nc * st.cg);
  group_means<kNT>(st, count, w, sums + int64_t(ch.sample) * 2 * channels, channels, ma, mb, sha, shb);
  const A* ss = stats + (int64_t(ch.sample) * num_groups + st.gid) * 2;
#define CALL(N) strip_grad<kNT, T, VEC, N, A>(st, p, ch.r0, ch.r1, x, g, gx, dim, w, b, ss, ma, mb, act)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
}

// A whole sample's strip by one workgroup: its channels' sums, then grad_x.
template <typename T, int VEC>
__global__ __launch_bounds__(kNTS) void norm_sample_grad_kernel(const int32_t* first_row, const NormStrip* strips,
                                                               int sample_first, Order ord, const T* x, const T* g,
                                                               T* gx, int64_t dim, int num_groups, int channels,
                                                               const T* w, const T* b,
                                                               const typename AccOf<T>::type* stats, int act,
                                                               typename AccOf<T>::type* sums) {
  using A = typename AccOf<T>::type;
  __shared__ A sh[kNTS][2 * VEC + 1];
  __shared__ A sha[kNTS], shb[kNTS], ma[kNTS], mb[kNTS];
  const int s = sample_first + ord.unit(), r0 = first_row[s], r1 = first_row[s + 1];
  const NormStrip st = ldc(strips + ord.strip());
  const Place p = place<VEC, kNTS>(st);
  const A* ss = stats + (int64_t(s) * num_groups + st.gid) * 2;
  A* o = sums + int64_t(s) * 2 * channels;
  // (an empty sample writes its zero sums)
#define CALL(N) strip_sums<kNTS, T, VEC, N, A>(st, p, r0, r1, x, g, dim, w, b, ss, act, o, channels, sh)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
  if (!gx || r0 == r1) return;
  const A count = A(r1 - r0) * A(st.nc * st.cg);
  group_means<kNTS>(st, count, w, o, channels, ma, mb, sha, shb);
#define CALL(N) strip_grad<kNTS, T, VEC, N, A>(st, p, r0, r1, x, g, gx, dim, w, b, ss, ma, mb, act)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// (at most kMaxWorkgroups: see slices; a single sample has at most 512 runs, and a
// norm some 6000 strips of 256 lanes)
Order strip_order(int64_t units, int nstrip) {
  return {int(units), nstrip, units * nstrip <= 1280};  // 5 workgroups a compute unit
}
dim3 strip_grid(const Order& o) { return dim3(unsigned(o.units * o.strips)); }

// The handle's lane width needs 16-byte aligned tensors and offsets that are
// multiples of it (every multiplicity is).
bool use_vec(const cgtp_norm_s* n, const void* a, const void* b, const void* c) {
  return n->vec > 1 && aligned16(a) && aligned16(b) && aligned16(c);
}

// f(integral constant VEC) for the lane width in use.
template <typename T, typename F>
void with_vec(int vec, F&& f) {
  constexpr int W = 16 / int(sizeof(T));
  if (vec == W) f(std::integral_constant<int, W>{});
  else if (W > 4 && vec == 4) f(std::integral_constant<int, W >= 4 ? 4 : 1>{});
  else if (W > 2 && vec == 2) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 1>{});
}

// Short samples (at most this many bytes of a narrow strip in a sample): one
// workgroup a sample and strip, one launch forward and two backward (96 samples of
// 20 - 220 rows 53 us, as runs 70 us; 8 molecules forward 8.9 us and 12.7 us). On
// both sides of the limit, bf16 rows of 1152, forward + backward in one graph, so /
// as runs: 32 samples of 128 KB 11 + 25 / 15 + 27 us, of 256 KB 18 + 34 / 21 + 43 us, of
// 512 KB 33 + 54 / 38 + 68 us; but 4 samples, which leave most of the device idle, of
// 128 KB 11 + 21 / 11 + 18 us, of 256 KB 14 + 27 / 11 + 18 us, of 1 MB 37 + 79 / 15 + 26 us.
constexpr int64_t kSampleBytes = 256 << 10;

bool by_sample(const cgtp_norm_s* n, const cgtp_samples_s* sm) {
  return sm->longest * n->narrow_row * int64_t(dtype_size(n->dtype)) <= kSampleBytes;
}

// Longer samples take two passes over the rows. The second reads them from the
// last-level cache if it follows soon enough, so the rows are worked off in
// slices of whole samples of about this many bytes a tensor (104,217 rows of 4 KB
// 270 us, all at once 315 us).
constexpr int64_t kSliceBytes = int64_t(160) << 20;

// f(first sample, end sample) for each slice; one launch takes a slice's runs of
// every strip, or its samples.
template <typename F>
void slices(const cgtp_samples_s* sm, int64_t row_bytes, int nstrip, F&& f) {
  const int64_t rows = std::max<int64_t>(1, kSliceBytes / row_bytes), most = kMaxWorkgroups / nstrip;
  const auto runs = [&](int64_t s) { return int64_t(sm->sample_chunk[size_t(s)]); };
  for (int64_t s = 0; s < sm->S;) {
    int64_t e = s + 1;
    while (e < sm->S && sm->ptr[size_t(e) + 1] - sm->ptr[size_t(s)] <= rows && runs(e + 1) - runs(s) <= most &&
           e + 1 - s <= kMaxWorkgroups)
      ++e;
    f(s, e);
    s = e;
  }
}

// f(first sample, end sample) for the launches that take whole samples.
template <typename F>
void sample_launches(int64_t S, int nstrip, F&& f) {
  const int64_t most = kMaxWorkgroups / nstrip;
  for (int64_t s = 0; s < S; s += most) f(s, std::min(s + most, S));
}

template <typename T>
void forward_typed(const cgtp_norm_s* n, const cgtp_samples_s* sm, const void* x, const void* w, const void* b,
                   void* y, void* stats, void* ws, hipStream_t s) {
  using A = typename AccOf<T>::type;
  if (sm->rows == 0) return;
  const bool v = use_vec(n, x, y, nullptr), one = by_sample(n, sm);
  const int kind = (v ? 0 : 1) + (one ? 2 : 0);
  const NormStrip* strips = n->strips[kind].as<NormStrip>();
  const int nstrip = n->nstrip[kind];
  const RowChunk* ch = sm->chunks.as<RowChunk>();
  const T *tx = static_cast<const T*>(x), *tw = static_cast<const T*>(w), *tb = static_cast<const T*>(b);
  T* ty = static_cast<T*>(y);
  auto* part = static_cast<Part<A>*>(ws);
  const int groups = int(n->num_groups);
  with_vec<T>(v ? n->vec : 1, [&](auto V) {
    if (one) {
      sample_launches(sm->S, nstrip, [&](int64_t s0, int64_t s1) {
        const Order order = strip_order(s1 - s0, nstrip);
        hipLaunchKernelGGL((norm_sample_kernel<T, V.value>), strip_grid(order), dim3(kNTS), 0, s,
                           sm->first_row.as<int32_t>(), strips, int(s0), order, tx, ty, n->row.dim, groups, tw, tb,
                           static_cast<A*>(stats), A(n->eps), int(n->act));
        CGTP_CHECK_HIP(hipGetLastError());
      });
      return;
    }
    slices(sm, n->row.dim * int64_t(sizeof(T)), nstrip, [&](int64_t s0, int64_t s1) {
      const int c0 = sm->sample_chunk[size_t(s0)], c1 = sm->sample_chunk[size_t(s1)];
      if (c0 == c1) return;  // empty samples
      const Order order = strip_order(c1 - c0, nstrip);
      const dim3 grid = strip_grid(order);
      hipLaunchKernelGGL((norm_moments_kernel<T, V.value>), grid, dim3(kNT), 0, s, ch, strips, tx, n->row.dim, groups,
                         c0, order, part);
      hipLaunchKernelGGL((norm_apply_kernel<T, V.value>), grid, dim3(kNT), 0, s, ch, strips, tx, ty, n->row.dim,
                         groups, c0, order, tw, tb, part, static_cast<A*>(stats), A(n->eps), int(n->act));
      CGTP_CHECK_HIP(hipGetLastError());
    });
  });
}

template <typename T>
void backward_typed(const cgtp_norm_s* n, const cgtp_samples_s* sm, const void* x, const void* w, const void* b,
                    const void* stats, const void* g, void* gx, void* gw, void* gb, void* ws, hipStream_t s) {
  using A = typename AccOf<T>::type;
  const int C = int(n->row.channels), groups = int(n->num_groups);
  if (sm->rows == 0) {
    if (gw) zero_rows(gw, n->row.channels, sizeof(T), s);
    if (gb && n->row.biases) zero_rows(gb, n->row.biases, sizeof(T), s);
    return;
  }
  const bool v = use_vec(n, x, g, gx), one = by_sample(n, sm);
  const int kind = (v ? 0 : 1) + (one ? 2 : 0);
  const NormStrip* strips = n->strips[kind].as<NormStrip>();
  const int nstrip = n->nstrip[kind];
  const RowChunk* ch = sm->chunks.as<RowChunk>();
  const T *tx = static_cast<const T*>(x), *tw = static_cast<const T*>(w), *tb = static_cast<const T*>(b);
  const T* tg = static_cast<const T*>(g);
  const A* st = static_cast<const A*>(stats);
  // per-sample sums [S][2][C], then the runs' [chunks][2][C]
  A* sums = static_cast<A*>(ws);
  A* part = sums + 2 * size_t(C) * size_t(sm->S);
  with_vec<T>(v ? n->vec : 1, [&](auto V) {
    if (one) {
      sample_launches(sm->S, nstrip, [&](int64_t s0, int64_t s1) {
        const Order order = strip_order(s1 - s0, nstrip);
        hipLaunchKernelGGL((norm_sample_grad_kernel<T, V.value>), strip_grid(order), dim3(kNTS), 0, s,
                           sm->first_row.as<int32_t>(), strips, int(s0), order, tx, tg, static_cast<T*>(gx),
                           n->row.dim, groups, C, tw, tb, st, int(n->act), sums);
        CGTP_CHECK_HIP(hipGetLastError());
      });
      return;
    }
    slices(sm, 2 * n->row.dim * int64_t(sizeof(T)), nstrip, [&](int64_t s0, int64_t s1) {
      const int c0 = sm->sample_chunk[size_t(s0)], c1 = sm->sample_chunk[size_t(s1)];
      const Order order = strip_order(c1 - c0, nstrip);
      const dim3 grid = strip_grid(order);
      if (c0 < c1)
        hipLaunchKernelGGL((norm_sums_kernel<T, V.value>), grid, dim3(kNT), 0, s, ch, strips, tx, tg, n->row.dim,
                           groups, C, c0, order, tw, tb, st, int(n->act), part);
      hipLaunchKernelGGL((norm_join_kernel<A>), dim3(unsigned(s1 - s0), unsigned((2 * C + 7) / 8)), dim3(kNT), 0, s,
                         sm->first.as<int32_t>(), int(s0), part, sums, 2 * C);
      if (gx && c0 < c1)
        hipLaunchKernelGGL((norm_grad_kernel<T, V.value>), grid, dim3(kNT), 0, s, ch, strips, tx, tg,
                           static_cast<T*>(gx), n->row.dim, groups, C, c0, order, tw, tb, st, sums, int(n->act));
      CGTP_CHECK_HIP(hipGetLastError());
    });
  });
  if (gw || gb) {
    hipLaunchKernelGGL((norm_param_kernel<T>), dim3(16, unsigned(nstrip)), dim3(kNT), 0, s, strips, sums, sm->S, C,
                       static_cast<T*>(gw), static_cast<T*>(gb));
    CGTP_CHECK_HIP(hipGetLastError());
  }
}

}  // namespace

size_t norm_ws_bytes(const cgtp_norm_s* n, const cgtp_samples_s* sm, bool backward) {
  const size_t es = acc_size(n->dtype);
  if (sm->rows == 0) return 0;
  const size_t runs = by_sample(n, sm) ? 0 : size_t(sm->nchunk);
  return backward ? (runs + size_t(sm->S)) * 2 * size_t(n->row.channels) * es : runs * size_t(n->num_groups) * 4 * es;
}

void norm_forward_launch(const cgtp_norm_s* n, const cgtp_samples_s* sm, const void* x, const void* w, const void* b,
                         void* y, void* stats, void* ws, hipStream_t s) {
  if (n->dtype == CGTP_F64) forward_typed<double>(n, sm, x, w, b, y, stats, ws, s);
  else if (n->dtype == CGTP_BF16) forward_typed<bf16>(n, sm, x, w, b, y, stats, ws, s);
  else forward_typed<float>(n, sm, x, w, b, y, stats, ws, s);
}

void norm_backward_launch(const cgtp_norm_s* n, const cgtp_samples_s* sm, const void* x, const void* w, const void* b,
                          const void* stats, const void* g, void* gx, void* gw, void* gb, void* ws, hipStream_t s) {
  if (n->dtype == CGTP_F64) backward_typed<double>(n, sm, x, w, b, stats, g, gx, gw, gb, ws, s);
  else if (n->dtype == CGTP_BF16) backward_typed<bf16>(n, sm, x, w, b, stats, g, gx, gw, gb, ws, s);
  else backward_typed<float>(n, sm, x, w, b, stats, g, gx, gw, gb, ws, s);
}

}  // namespace cgtp
