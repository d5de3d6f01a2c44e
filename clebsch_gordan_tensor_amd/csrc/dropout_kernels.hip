// Dropout on irreps rows from a counter-based generator, with an optional
// residual added in the same pass.
//
// y = residual + (draw >= t ? x * 65536 / (65536 - t) : 0), one 16-bit draw per
// channel, shared by its 2l+1 components (the mask then commutes with
// rotations). Draws: Philox 4x32, 10 rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011); one evaluation yields
// 128 bits = the draws of 8 channels, which is one 16-byte bf16 access.
//
// Bound: memory (x and residual read, y written once). A thread takes 8
// channels of one row and all their components, so one generator evaluation
// (about 20 wide multiplies) serves 8 (2l+1) elements and runs while the loads
// are in flight. A workgroup handles one block, so that every lane of a wave
// has the same component count and neighbouring lanes read neighbouring 16-byte
// pieces of a component's channels.
#include <algorithm>

#include "device_util.hpp"
#include "layers.hpp"

namespace cgtp {

namespace {

constexpr int kDropThreads = 256;

struct Draws {
  uint32_t w[4];
};

__device__ __forceinline__ Draws philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                        uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    const uint32_t n0 = uint32_t(b >> 32) ^ c1 ^ k0, n2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c1 = uint32_t(b);
    c3 = uint32_t(a);
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// 8 consecutive elements as 16-byte accesses.
template <typename T, typename A>
__device__ __forceinline__ void load8(const T* p, A (&o)[8]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int k = 0; k < 8; k += V) {
    A t[V];
    VecIO<T, V>::load(p + k, t);
#pragma unroll
    for (int i = 0; i < V; ++i) o[k + i] = t[i];
  }
}

// Stored past the caches: results are not read again soon (2^18 rows of 4 KB,
// forward and backward: 1105 us against 1191 us; with rows at a time and a grid of
// at most 4096 row groups 1005 us = 5.3 TB/s).
template <typename T, typename A>
__device__ __forceinline__ void store8(T* p, const A (&o)[8]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int k = 0; k < 8; k += V) {
    A t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = o[k + i];
    VecIO<T, V>::store_nt(p + k, t);
  }
}

struct DropArgs {
  int64_t B, dim;
  uint32_t k0, k1, offset, t;
};

// One block of NC components; RES: a residual is added; WIDE: 16-byte accesses.
template <typename T, int NC, bool RES, bool WIDE>
__device__ __forceinline__ void drop_block(const RowBlock& b, const DropArgs& a, const T* x, const T* res,
                                           T* y, typename AccOf<T>::type scale) {
  using A = typename AccOf<T>::type;
  const int nch = (b.mul + 7) / 8;  // chunks of the block
  const int per_row = nch < kDropThreads ? nch : kDropThreads;
  const int rows_per_pass = kDropThreads / per_row;
  const int slot = int(threadIdx.x) / per_row, first = int(threadIdx.x) % per_row;
  if (slot >= rows_per_pass) return;
  const int64_t step = int64_t(gridDim.x) * rows_per_pass;
  if constexpr (WIDE) {
    // rows at a time, so that the narrow blocks have some accesses in flight too
    constexpr int RU = NC == 1 ? 4 : NC == 3 ? 2 : 1;
    for (int64_t r = int64_t(blockIdx.x) * rows_per_pass + slot; r < a.B; r += RU * step)
      for (int c = first; c < nch; c += per_row) {
        A v[RU][NC][8], q[RES ? RU : 1][RES ? NC : 1][8];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          const int64_t at = min(r + u * step, a.B - 1) * a.dim + b.off + 8 * c;
#pragma unroll
          for (int m = 0; m < NC; ++m) {
            load8(x + at + m * b.mul, v[u][m]);
            if constexpr (RES) load8(res + at + m * b.mul, q[u][m]);
          }
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          const int64_t row = r + u * step, at = row * a.dim + b.off + 8 * c;
          if (row >= a.B) break;
          const Draws d =
              philox(uint32_t(b.chunk + c), uint32_t(row), uint32_t(uint64_t(row) >> 32), a.offset, a.k0, a.k1);
#pragma unroll
          for (int m = 0; m < NC; ++m) {
            A o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t draw = (i & 1) ? d.w[i / 2] >> 16 : d.w[i / 2] & 0xffffu;
              o[i] = draw >= a.t ? v[u][m][i] * scale : A(0);
              if constexpr (RES) o[i] += q[u][m][i];
            }
            store8(y + at + m * b.mul, o);
          }
        }
      }
  } else {
    for (int64_t r = int64_t(blockIdx.x) * rows_per_pass + slot; r < a.B; r += step)
      for (int c = first; c < nch; c += per_row) {
        const int64_t at = r * a.dim + b.off + 8 * c;
        const Draws d = philox(uint32_t(b.chunk + c), uint32_t(r), uint32_t(uint64_t(r) >> 32), a.offset, a.k0, a.k1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (8 * c + i >= b.mul) break;
          const uint32_t draw = (i & 1) ? d.w[i / 2] >> 16 : d.w[i / 2] & 0xffffu;
#pragma unroll
          for (int m = 0; m < NC; ++m) {
            const int64_t e = at + m * b.mul + i;
            A o = draw >= a.t ? to_acc<A>(x[e]) * scale : A(0);
            if (RES) o += to_acc<A>(res[e]);
            from_acc(y[e], o);
          }
        }
      }
  }
}

template <typename T, bool RES, bool WIDE>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(const RowBlock* blocks, DropArgs a, const T* x,
                                                               const T* res, T* y, typename AccOf<T>::type scale) {
  const RowBlock b = ldc(blocks + blockIdx.y);
  switch (b.nc) {
    case 1: drop_block<T, 1, RES, WIDE>(b, a, x, res, y, scale); break;
    case 3: drop_block<T, 3, RES, WIDE>(b, a, x, res, y, scale); break;
    case 5: drop_block<T, 5, RES, WIDE>(b, a, x, res, y, scale); break;
    case 7: drop_block<T, 7, RES, WIDE>(b, a, x, res, y, scale); break;
    default: drop_block<T, 9, RES, WIDE>(b, a, x, res, y, scale); break;
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T>
void launch_typed(const cgtp_dropout_s* d, const DropArgs& a, const void* x, const void* residual, void* y,
                  hipStream_t s) {
  using A = typename AccOf<T>::type;
  bool wide = aligned16(x) && aligned16(residual) && aligned16(y);
  int64_t per_row = kDropThreads;
  for (const RowBlock& b : d->row.blocks) {
    wide = wide && b.mul % 8 == 0;
    per_row = std::min<int64_t>(per_row, (b.mul + 7) / 8);
  }
  const int64_t passes = (a.B * per_row + kDropThreads - 1) / kDropThreads;  // of the narrowest block
  const dim3 grid(unsigned(std::max<int64_t>(1, std::min<int64_t>(passes, 4096))), unsigned(d->row.blocks.size()));
  const A scale = A(65536.0 / (65536.0 - double(a.t)));
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kDropThreads), 0, s, d->blocks.as<RowBlock>(), a, static_cast<const T*>(x),
                       static_cast<const T*>(residual), static_cast<T*>(y), scale);
  };
  if (residual) {
    if (wide) go(dropout_kernel<T, true, true>);
    else go(dropout_kernel<T, true, false>);
  } else {
    if (wide) go(dropout_kernel<T, false, true>);
    else go(dropout_kernel<T, false, false>);
  }
  CGTP_CHECK_HIP(hipGetLastError());
}

}  // namespace

void dropout_launch(const cgtp_dropout_s* d, int64_t B, const void* x, double p, uint64_t seed, uint32_t offset,
                    const void* residual, void* y, hipStream_t s) {
  DropArgs a{};
  a.B = B;
  a.dim = d->row.dim;
  a.k0 = uint32_t(seed);
  a.k1 = uint32_t(seed >> 32);
  a.offset = offset;
  a.t = std::min<uint32_t>(65535u, uint32_t(p * 65536.0 + 0.5));
  if (d->dtype == CGTP_F64)
    launch_typed<double>(d, a, x, residual, y, s);
  else if (d->dtype == CGTP_BF16)
    launch_typed<bf16>(d, a, x, residual, y, s);
  else
    launch_typed<float>(d, a, x, residual, y, s);
}

}  // namespace cgtp
