// Cross attention kernels, bf16, padded head sizes 32, 64, 96, 128.
#include "attn_impl.hpp"

namespace cgtp {
namespace attn {

KernelTable kernels_bf16_a(int dp) {
  switch (dp) {
    case 32: return Kernels<bf16, 32>::table();
    case 64: return Kernels<bf16, 64>::table();
    case 96: return Kernels<bf16, 96>::table();
    default: return Kernels<bf16, 128>::table();
  }
}

}  // namespace attn
}  // namespace cgtp
