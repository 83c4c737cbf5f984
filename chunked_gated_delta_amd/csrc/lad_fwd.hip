// The outputs of linear attention with a decay for each head, and its final states.
#include "lad_walk.h"

namespace kda {

hipError_t launch_lad_fwd(const LadParams& p, int dtype, int dx, int dz, hipStream_t s) {
  if (dtype == KDA_DTYPE_BF16 && !p.walk[0].leaving) return launch_walk_dims<uint16_t, 2, 2, lad::kOuts>(p, dx, dz, s);
  return dtype == KDA_DTYPE_BF16 ? launch_walk_dims<uint16_t, 3, 2, lad::kOuts>(p, dx, dz, s) : launch_walk_dims<float, 3, 2, lad::kOuts>(p, dx, dz, s);
}

}  // namespace kda
