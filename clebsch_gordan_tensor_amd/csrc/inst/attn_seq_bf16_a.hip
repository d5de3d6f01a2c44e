// Kernels of attention along sequences, bf16, padded head sizes 32, 64, 96, 128.
#include "attn_seq_impl.hpp"

namespace cgtp {
namespace attn {

SeqTable seq_kernels_bf16_a(int dp) {
  switch (dp) {
    case 32: return SeqKernels<bf16, 32>::table();
    case 64: return SeqKernels<bf16, 64>::table();
    case 96: return SeqKernels<bf16, 96>::table();
    default: return SeqKernels<bf16, 128>::table();
  }
}

}  // namespace attn
}  // namespace cgtp
