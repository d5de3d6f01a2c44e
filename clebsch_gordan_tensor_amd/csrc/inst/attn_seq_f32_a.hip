// Kernels of attention along sequences, f32, padded head sizes 32, 64, 96, 128.
#include "attn_seq_impl.hpp"

namespace cgtp {
namespace attn {

SeqTable seq_kernels_f32_a(int dp) {
  switch (dp) {
    case 32: return SeqKernels<float, 32>::table();
    case 64: return SeqKernels<float, 64>::table();
    case 96: return SeqKernels<float, 96>::table();
    default: return SeqKernels<float, 128>::table();
  }
}

}  // namespace attn
}  // namespace cgtp
