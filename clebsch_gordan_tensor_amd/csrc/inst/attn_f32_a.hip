// Cross attention kernels, f32, padded head sizes 32, 64, 96, 128.
#include "attn_impl.hpp"

namespace cgtp {
namespace attn {

KernelTable kernels_f32_a(int dp) {
  switch (dp) {
    case 32: return Kernels<float, 32>::table();
    case 64: return Kernels<float, 64>::table();
    case 96: return Kernels<float, 96>::table();
    default: return Kernels<float, 128>::table();
  }
}

}  // namespace attn
}  // namespace cgtp
