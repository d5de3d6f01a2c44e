// Kernels of attention along sequences, f32, padded head sizes 160, 192, 224, 256.
#include "attn_seq_impl.hpp"

namespace cgtp {
namespace attn {

SeqTable seq_kernels_f32_b(int dp) {
  switch (dp) {
    case 160: return SeqKernels<float, 160>::table();
    case 192: return SeqKernels<float, 192>::table();
    case 224: return SeqKernels<float, 224>::table();
    default: return SeqKernels<float, 256>::table();
  }
}

}  // namespace attn
}  // namespace cgtp
