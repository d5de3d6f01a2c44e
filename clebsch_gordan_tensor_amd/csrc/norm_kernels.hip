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
#include "device_util.hpp"
#include "layers.hpp"

namespace cgtp {

namespace {

constexpr int kNT = 256;

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
template <int VEC>
__device__ __forceinline__ Place place(const NormStrip& st) {
  Place p;
  p.lanes = st.ng * st.cg / VEC;
  p.per = p.lanes < kNT ? p.lanes : kNT;
  p.slots = kNT / p.per;
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
__device__ __forceinline__ Moments<A> merge(const Moments<A>& a, const Moments<A>& b) {
  const A n = a.n + b.n;
  if (!(n > A(0))) return a;
  const A d = b.mean - a.mean, f = b.n / n;
  return {n, a.mean + d * f, a.m2 + b.m2 + d * d * a.n * f};
}

// Rows kept in flight by a thread: about 8 accesses.
template <int NC>
struct RowsAhead {
  static constexpr int value = NC >= 5 ? 1 : (NC == 3 ? 2 : 4);
};

// Moments of the thread's elements of channel vector `lane0`.
template <typename T, int VEC, int NC, typename A = typename AccOf<T>::type>
__device__ __forceinline__ Moments<A> thread_moments(const NormStrip& st, const Place& p, int lane0, int r0, int r1,
                                                     const T* x, int64_t dim) {
  constexpr int RU = RowsAhead<NC>::value;
  const bool even = st.bias >= 0;
  const T* base = x + st.off + p.chan0 + lane0 * VEC;
  A s1 = 0, s2 = 0, pivot = 0;
  int64_t n = 0;
  if (r0 + p.slot < r1 && even) pivot = to_acc<A>(base[int64_t(r0 + p.slot) * dim]);
  for (int r = r0 + p.slot; r < r1; r += p.slots * RU) {
    A v[RU][NC][VEC];
#pragma unroll
    for (int u = 0; u < RU; ++u)
      if (r + u * p.slots < r1)
#pragma unroll
        for (int m = 0; m < NC; ++m)
          VecIO<T, VEC>::load(base + int64_t(r + u * p.slots) * dim + m * st.mul, v[u][m]);
#pragma unroll
    for (int u = 0; u < RU; ++u)
      if (r + u * p.slots < r1) {
        n += NC * VEC;
#pragma unroll
        for (int m = 0; m < NC; ++m)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const A d = v[u][m][i] - pivot;
            s1 += d;
            s2 += d * d;
          }
      }
  }
  if (n == 0) return {A(0), A(0), A(0)};
  if (!even) return {A(n), A(0), s2};
  const A f = s1 / A(n);
  const A m2 = s2 - s1 * f;
  return {A(n), pivot + f, m2 > A(0) || m2 != m2 ? m2 : A(0)};
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

template <int VEC>
__device__ __forceinline__ int lanes_of_group(const NormStrip& st, const Place& p) {
  return p.lanes > kNT ? kNT : st.cg / VEC;
}

// Moments of the groups of one strip over rows r0 .. r1, left in sh.
template <typename T, int VEC, int NC, typename A>
__device__ __forceinline__ void strip_moments(const NormStrip& st, const Place& p, int r0, int r1, const T* x,
                                              int64_t dim, Moments<A>* sh) {
  Moments<A> t{A(0), A(0), A(0)};
  if (p.slot < p.slots)
    for (int l = p.lane; l < p.lanes; l += kNT) t = merge(t, thread_moments<T, VEC, NC>(st, p, l, r0, r1, x, dim));
  sh[threadIdx.x] = t;
  group_tree(sh, p, lanes_of_group<VEC>(st, p));
}

#define CGTP_NC_SWITCH(nc, CALL) \
  switch (nc) {                  \
    case 1: CALL(1); break;      \
    case 3: CALL(3); break;      \
    case 5: CALL(5); break;      \
    case 7: CALL(7); break;      \
    default: CALL(9); break;     \
  }

// Mean and centred square sum of every group over one run of rows:
// part [chunk][groups][2].
template <typename T, int VEC>
__global__ __launch_bounds__(kNT) void norm_moments_kernel(const RowChunk* chunks, const NormStrip* strips, const T* x,
                                                           int64_t dim, int num_groups,
                                                           typename AccOf<T>::type* part) {
  using A = typename AccOf<T>::type;
  __shared__ Moments<A> sh[kNT];
  const RowChunk ch = ldc(chunks + blockIdx.x);
  const NormStrip st = ldc(strips + blockIdx.y);
  const Place p = place<VEC>(st);
#define CALL(N) strip_moments<T, VEC, N, A>(st, p, ch.r0, ch.r1, x, dim, sh)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
  const int lg = lanes_of_group<VEC>(st, p);
  if (int(threadIdx.x) < st.ng) {
    const Moments<A> g = sh[threadIdx.x * lg];
    A* o = part + (int64_t(blockIdx.x) * num_groups + st.gid + threadIdx.x) * 2;
    o[0] = g.mean;
    o[1] = g.m2;
  }
}

// y of the thread's channels over rows r0 .. r1 from the group's mean and rstd.
template <typename T, int VEC, int NC, typename A>
__device__ __forceinline__ void strip_apply(const NormStrip& st, const Place& p, int r0, int r1, const T* x, T* y,
                                            int64_t dim, const T* w, const T* b, const A* mean, const A* rstd,
                                            int act) {
  constexpr int RU = RowsAhead<NC>::value;
  if (p.slot >= p.slots) return;
  for (int l = p.lane; l < p.lanes; l += kNT) {
    const int c0 = p.chan0 + l * VEC, g = l * VEC / st.cg;
    const A mu = mean[g], r0s = rstd[g];
    A a[VEC], sft[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      a[i] = w ? r0s * to_acc<A>(w[st.chan + c0 + i]) : r0s;
      sft[i] = st.bias >= 0 && b ? to_acc<A>(b[st.bias + c0 + i]) : A(0);
    }
    const int on = NC == 1 && st.bias >= 0 ? act : int(CGTP_ACT_NONE);
    const int64_t at = st.off + c0;
    for (int r = r0 + p.slot; r < r1; r += p.slots * RU) {
      A v[RU][NC][VEC];
#pragma unroll
      for (int u = 0; u < RU; ++u)
        if (r + u * p.slots < r1)
#pragma unroll
          for (int m = 0; m < NC; ++m)
            VecIO<T, VEC>::load(x + int64_t(r + u * p.slots) * dim + at + m * st.mul, v[u][m]);
#pragma unroll
      for (int u = 0; u < RU; ++u)
        if (r + u * p.slots < r1)
#pragma unroll
          for (int m = 0; m < NC; ++m) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const A z = (v[u][m][i] - mu) * a[i] + sft[i];
              v[u][m][i] = NC == 1 ? act_value(on, z) : z;
            }
            VecIO<T, VEC>::store(y + int64_t(r + u * p.slots) * dim + at + m * st.mul, v[u][m]);
          }
    }
  }
}

// Joins the runs' moments of a sample's groups and writes y of one run.
template <typename T, int VEC>
__global__ __launch_bounds__(kNT) void norm_apply_kernel(const RowChunk* chunks, const NormStrip* strips, const T* x,
                                                         T* y, int64_t dim, int num_groups, const T* w, const T* b,
                                                         const typename AccOf<T>::type* part,
                                                         typename AccOf<T>::type* stats,
                                                         typename AccOf<T>::type eps, int act) {
  using A = typename AccOf<T>::type;
  __shared__ Moments<A> sh[kNT];
  __shared__ A mean[kNT], rstd[kNT];
  const RowChunk ch = ldc(chunks + blockIdx.x);
  const NormStrip st = ldc(strips + blockIdx.y);
  const Place p = place<VEC>(st);
  // kNT / ng threads a group, each a fixed part of the runs
  Place q;
  q.per = st.ng;
  q.slots = kNT / st.ng;
  q.slot = int(threadIdx.x) / st.ng;
  q.lane = int(threadIdx.x) % st.ng;
  q.lanes = q.chan0 = 0;
  Moments<A> t{A(0), A(0), A(0)};
  if (q.slot < q.slots)
    for (int k = q.slot; k < ch.nchunk; k += q.slots) {
      const RowChunk o = chunks[ch.chunk0 + k];
      const A* m = part + (int64_t(ch.chunk0 + k) * num_groups + st.gid + q.lane) * 2;
      t = merge(t, Moments<A>{A(o.r1 - o.r0) * A(st.nc * st.cg), m[0], m[1]});
    }
  sh[threadIdx.x] = t;
  group_tree(sh, q, 1);
  if (int(threadIdx.x) < st.ng) {
    const Moments<A> g = sh[threadIdx.x];
    const A r = rsqrt_acc(g.m2 / g.n + eps);
    mean[threadIdx.x] = g.mean;
    rstd[threadIdx.x] = r;
    if (stats && ch.r0 == ch.row0) {
      A* o = stats + (int64_t(ch.sample) * num_groups + st.gid + threadIdx.x) * 2;
      o[0] = g.mean;
      o[1] = r;
    }
  }
  __syncthreads();
#define CALL(N) strip_apply<T, VEC, N, A>(st, p, ch.r0, ch.r1, x, y, dim, w, b, mean, rstd, act)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
}

// A_c and B_c of one run of rows: part [chunk][2][channels].
template <typename T, int VEC, int NC, typename A>
__device__ __forceinline__ void strip_sums(const NormStrip& st, const Place& p, const RowChunk& ch, const T* x,
                                           const T* g, int64_t dim, const T* w, const T* b, const A* stats, int act,
                                           A* part, int channels, A (*sh)[2 * VEC]) {
  constexpr int RU = NC == 1 ? 2 : 1;
  for (int l0 = 0; l0 < p.lanes; l0 += kNT) {
    const int l = l0 + p.lane;
    A sa[VEC], sb[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) sa[i] = sb[i] = A(0);
    const int c0 = p.chan0 + l * VEC;
    if (p.slot < p.slots && l < p.lanes) {
      const int gi = l * VEC / st.cg;
      const A mu = stats[2 * gi], r0s = stats[2 * gi + 1];
      A wv[VEC], bv[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        wv[i] = w ? to_acc<A>(w[st.chan + c0 + i]) : A(1);
        bv[i] = st.bias >= 0 && b ? to_acc<A>(b[st.bias + c0 + i]) : A(0);
      }
      const int on = NC == 1 && st.bias >= 0 ? act : int(CGTP_ACT_NONE);
      const int64_t at = st.off + c0;
      for (int r = ch.r0 + p.slot; r < ch.r1; r += p.slots * RU) {
        A v[RU][NC][VEC], d[RU][NC][VEC];
#pragma unroll
        for (int u = 0; u < RU; ++u)
          if (r + u * p.slots < ch.r1)
#pragma unroll
            for (int m = 0; m < NC; ++m) {
              const int64_t e = int64_t(r + u * p.slots) * dim + at + m * st.mul;
              VecIO<T, VEC>::load(x + e, v[u][m]);
              VecIO<T, VEC>::load(g + e, d[u][m]);
            }
#pragma unroll
        for (int u = 0; u < RU; ++u)
          if (r + u * p.slots < ch.r1)
#pragma unroll
            for (int m = 0; m < NC; ++m)
#pragma unroll
              for (int i = 0; i < VEC; ++i) {
                const A xh = (v[u][m][i] - mu) * r0s;
                const A gz = NC == 1 ? d[u][m][i] * act_slope(on, xh * wv[i] + bv[i]) : d[u][m][i];
                sa[i] += gz * xh;
                sb[i] += gz;
              }
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      sh[threadIdx.x][i] = sa[i];
      sh[threadIdx.x][VEC + i] = sb[i];
    }
    __syncthreads();
    for (int cur = p.slots; cur > 1;) {
      const int half = (cur + 1) / 2;
      if (p.slot + half < cur)
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) sh[threadIdx.x][i] += sh[threadIdx.x + half * p.per][i];
      cur = half;
      __syncthreads();
    }
    if (p.slot == 0 && l < p.lanes)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        part[st.chan + c0 + i] = sh[threadIdx.x][i];
        part[channels + st.chan + c0 + i] = sh[threadIdx.x][VEC + i];
      }
    __syncthreads();
  }
}

template <typename T, int VEC>
__global__ __launch_bounds__(kNT) void norm_sums_kernel(const RowChunk* chunks, const NormStrip* strips, const T* x,
                                                        const T* g, int64_t dim, int num_groups, int channels,
                                                        const T* w, const T* b, const typename AccOf<T>::type* stats,
                                                        int act, typename AccOf<T>::type* part) {
  using A = typename AccOf<T>::type;
  __shared__ A sh[kNT][2 * VEC];
  const RowChunk ch = ldc(chunks + blockIdx.x);
  const NormStrip st = ldc(strips + blockIdx.y);
  const Place p = place<VEC>(st);
  const A* ss = stats + (int64_t(ch.sample) * num_groups + st.gid) * 2;
  A* o = part + int64_t(blockIdx.x) * 2 * channels;
#define CALL(N) strip_sums<T, VEC, N, A>(st, p, ch, x, g, dim, w, b, ss, act, o, channels, sh)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
}

// Sums rows first[s] .. first[s + 1] of part [chunk][cols] into out [s][cols]:
// 16 columns and 16 rows at a time, fixed order.
template <typename A>
__global__ __launch_bounds__(kNT) void norm_join_kernel(const int32_t* first, const A* part, A* out, int cols) {
  __shared__ A sh[16][17];
  const int s = blockIdx.x, c = int(blockIdx.y) * 16 + int(threadIdx.x) % 16, j = int(threadIdx.x) / 16;
  A t = 0;
  if (c < cols)
    for (int k = first[s] + j; k < first[s + 1]; k += 16) t += part[int64_t(k) * cols + c];
  sh[j][threadIdx.x % 16] = t;
  __syncthreads();
  if (j == 0 && c < cols) {
    for (int k = 1; k < 16; ++k) t += sh[k][threadIdx.x];
    out[int64_t(s) * cols + c] = t;
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
template <typename T, int VEC, int NC, typename A>
__device__ __forceinline__ void strip_grad(const NormStrip& st, const Place& p, int r0, int r1, const T* x, const T* g,
                                           T* gx, int64_t dim, const T* w, const T* b, const A* stats, const A* mean_a,
                                           const A* mean_b, int act) {
  constexpr int RU = NC == 1 ? 2 : 1;
  if (p.slot >= p.slots) return;
  for (int l = p.lane; l < p.lanes; l += kNT) {
    const int c0 = p.chan0 + l * VEC, gi = l * VEC / st.cg;
    const A mu = stats[2 * gi], r0s = stats[2 * gi + 1], ma = mean_a[gi], mb = mean_b[gi];
    A wv[VEC], bv[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      wv[i] = w ? to_acc<A>(w[st.chan + c0 + i]) : A(1);
      bv[i] = st.bias >= 0 && b ? to_acc<A>(b[st.bias + c0 + i]) : A(0);
    }
    const int on = NC == 1 && st.bias >= 0 ? act : int(CGTP_ACT_NONE);
    const int64_t at = st.off + c0;
    for (int r = r0 + p.slot; r < r1; r += p.slots * RU) {
      A v[RU][NC][VEC], d[RU][NC][VEC];
#pragma unroll
      for (int u = 0; u < RU; ++u)
        if (r + u * p.slots < r1)
#pragma unroll
          for (int m = 0; m < NC; ++m) {
            const int64_t e = int64_t(r + u * p.slots) * dim + at + m * st.mul;
            VecIO<T, VEC>::load(x + e, v[u][m]);
            VecIO<T, VEC>::load(g + e, d[u][m]);
          }
#pragma unroll
      for (int u = 0; u < RU; ++u)
        if (r + u * p.slots < r1)
#pragma unroll
          for (int m = 0; m < NC; ++m) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const A xh = (v[u][m][i] - mu) * r0s;
              const A gz = NC == 1 ? d[u][m][i] * act_slope(on, xh * wv[i] + bv[i]) : d[u][m][i];
              v[u][m][i] = r0s * (gz * wv[i] - mb - xh * ma);
            }
            VecIO<T, VEC>::store(gx + int64_t(r + u * p.slots) * dim + at + m * st.mul, v[u][m]);
          }
    }
  }
}

// Means of w A and w B over the groups of a strip, from per-channel sums.
template <int VEC, typename T, typename A>
__device__ __forceinline__ void group_means(const NormStrip& st, A count, const T* w, const A* sums, int channels,
                                            A* mean_a, A* mean_b, A* sha, A* shb) {
  // kNT / ng threads a group (ng <= kNT); fixed order
  const int slots = kNT / st.ng, slot = int(threadIdx.x) / st.ng, gi = int(threadIdx.x) % st.ng;
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
                                                        const T* w, const T* b, const typename AccOf<T>::type* stats,
                                                        const typename AccOf<T>::type* sums, int act) {
  using A = typename AccOf<T>::type;
  __shared__ A sha[kNT], shb[kNT], ma[kNT], mb[kNT];
  const RowChunk ch = ldc(chunks + blockIdx.x);
  const NormStrip st = ldc(strips + blockIdx.y);
  const Place p = place<VEC>(st);
  const A count = A(ch.rows) * A(st.nc * st.cg);
  group_means<VEC>(st, count, w, sums + int64_t(ch.sample) * 2 * channels, channels, ma, mb, sha, shb);
  const A* ss = stats + (int64_t(ch.sample) * num_groups + st.gid) * 2;
#define CALL(N) strip_grad<T, VEC, N, A>(st, p, ch.r0, ch.r1, x, g, gx, dim, w, b, ss, ma, mb, act)
  CGTP_NC_SWITCH(st.nc, CALL)
#undef CALL
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

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

template <typename T>
void forward_typed(const cgtp_norm_s* n, const cgtp_samples_s* sm, const void* x, const void* w, const void* b,
                   void* y, void* stats, void* ws, hipStream_t s) {
  using A = typename AccOf<T>::type;
  if (sm->rows == 0) return;
  const bool v = use_vec(n, x, y, nullptr);
  const NormStrip* strips = n->strips[v ? 0 : 1].as<NormStrip>();
  const dim3 grid(unsigned(sm->nchunk), unsigned(n->nstrip[v ? 0 : 1]));
  const RowChunk* ch = sm->chunks.as<RowChunk>();
  A* part = static_cast<A*>(ws);
  with_vec<T>(v ? n->vec : 1, [&](auto V) {
    hipLaunchKernelGGL((norm_moments_kernel<T, V.value>), grid, dim3(kNT), 0, s, ch, strips, static_cast<const T*>(x),
                       n->row.dim, int(n->num_groups), part);
    CGTP_CHECK_HIP(hipGetLastError());
    hipLaunchKernelGGL((norm_apply_kernel<T, V.value>), grid, dim3(kNT), 0, s, ch, strips, static_cast<const T*>(x),
                       static_cast<T*>(y), n->row.dim, int(n->num_groups), static_cast<const T*>(w),
                       static_cast<const T*>(b), part, static_cast<A*>(stats), A(n->eps), int(n->act));
    CGTP_CHECK_HIP(hipGetLastError());
  });
}

template <typename T>
void backward_typed(const cgtp_norm_s* n, const cgtp_samples_s* sm, const void* x, const void* w, const void* b,
                    const void* stats, const void* g, void* gx, void* gw, void* gb, void* ws, hipStream_t s) {
  using A = typename AccOf<T>::type;
  const int C = int(n->row.channels);
  if (sm->rows == 0) {
    if (gw) zero_rows(gw, n->row.channels, sizeof(T), s);
    if (gb && n->row.biases) zero_rows(gb, n->row.biases, sizeof(T), s);
    return;
  }
  const bool v = use_vec(n, x, g, gx);
  const NormStrip* strips = n->strips[v ? 0 : 1].as<NormStrip>();
  const int nstrip = n->nstrip[v ? 0 : 1];
  const dim3 grid(unsigned(sm->nchunk), unsigned(nstrip));
  const RowChunk* ch = sm->chunks.as<RowChunk>();
  A* part = static_cast<A*>(ws);
  A* sums = part + 2 * size_t(C) * size_t(sm->nchunk);
  with_vec<T>(v ? n->vec : 1, [&](auto V) {
    hipLaunchKernelGGL((norm_sums_kernel<T, V.value>), grid, dim3(kNT), 0, s, ch, strips, static_cast<const T*>(x),
                       static_cast<const T*>(g), n->row.dim, int(n->num_groups), C, static_cast<const T*>(w),
                       static_cast<const T*>(b), static_cast<const A*>(stats), int(n->act), part);
    CGTP_CHECK_HIP(hipGetLastError());
    hipLaunchKernelGGL((norm_join_kernel<A>), dim3(unsigned(sm->S), unsigned((2 * C + 15) / 16)), dim3(kNT), 0, s,
                       sm->first.as<int32_t>(), part, sums, 2 * C);
    CGTP_CHECK_HIP(hipGetLastError());
    if (gx) {
      hipLaunchKernelGGL((norm_grad_kernel<T, V.value>), grid, dim3(kNT), 0, s, ch, strips, static_cast<const T*>(x),
                         static_cast<const T*>(g), static_cast<T*>(gx), n->row.dim, int(n->num_groups), C,
                         static_cast<const T*>(w), static_cast<const T*>(b), static_cast<const A*>(stats), sums,
                         int(n->act));
      CGTP_CHECK_HIP(hipGetLastError());
    }
  });
  if (gw || gb) {
    hipLaunchKernelGGL((norm_param_kernel<T>), dim3(16, unsigned(nstrip)), dim3(kNT), 0, s, strips, sums, sm->S, C,
                       static_cast<T*>(gw), static_cast<T*>(gb));
    CGTP_CHECK_HIP(hipGetLastError());
  }
}

}  // namespace

size_t norm_ws_bytes(const cgtp_norm_s* n, const cgtp_samples_s* sm) {
  const size_t es = acc_size(n->dtype), nch = size_t(sm->nchunk);
  const size_t fwd = nch * size_t(n->num_groups) * 2 * es;
  const size_t bwd = (nch + size_t(sm->S)) * 2 * size_t(n->row.channels) * es;
  return sm->rows == 0 ? 0 : std::max(fwd, bwd);
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
