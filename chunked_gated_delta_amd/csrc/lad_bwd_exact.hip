// The gradients of q, k and v where a decay's gradient in fp32 is taken from them, and in fp32.
#include "lad_walk.h"

namespace kda {

hipError_t launch_lad_bwd_exact(const LadParams& p, int dtype, int dx, int dz, hipStream_t s) {
  return dtype == KDA_DTYPE_BF16 ? launch_walk_dims<uint16_t, 3, 3, lad::kParts>(p, dx, dz, s) : launch_walk_dims<float, 3, 3, lad::kDots>(p, dx, dz, s);
}

}  // namespace kda
