// Cross attention kernels, f32, padded head sizes 160, 192, 224, 256.
#include "attn_impl.hpp"

namespace cgtp {
namespace attn {

KernelTable kernels_f32_b(int dp) {
  switch (dp) {
    case 160: return Kernels<float, 160>::table();
    case 192: return Kernels<float, 192>::table();
    case 224: return Kernels<float, 224>::table();
    default: return Kernels<float, 256>::table();
  }
}

}  // namespace attn
}  // namespace cgtp
