// Kernels of attention along sequences, bf16, padded head sizes 160, 192, 224, 256.
#include "attn_seq_impl.hpp"

namespace cgtp {
namespace attn {

SeqTable seq_kernels_bf16_b(int dp) {
  switch (dp) {
    case 160: return SeqKernels<bf16, 160>::table();
    case 192: return SeqKernels<bf16, 192>::table();
    case 224: return SeqKernels<bf16, 224>::table();
    default: return SeqKernels<bf16, 256>::table();
  }
}

}  // namespace attn
}  // namespace cgtp
