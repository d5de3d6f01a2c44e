// Cross attention kernels, bf16, padded head sizes 160, 192, 224, 256.
#include "attn_impl.hpp"

namespace cgtp {
namespace attn {

KernelTable kernels_bf16_b(int dp) {
  switch (dp) {
    case 160: return Kernels<bf16, 160>::table();
    case 192: return Kernels<bf16, 192>::table();
    case 224: return Kernels<bf16, 224>::table();
    default: return Kernels<bf16, 256>::table();
  }
}

}  // namespace attn
}  // namespace cgtp
