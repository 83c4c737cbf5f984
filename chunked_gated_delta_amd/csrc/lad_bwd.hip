// The gradients of q, k and v in bf16: the walk over other tensors, its states only entering results in bf16.
#include "lad_walk.h"

namespace kda {

hipError_t launch_lad_bwd(const LadParams& p, int dtype, int dx, int dz, bool exact, hipStream_t s) {
  if (dtype == KDA_DTYPE_F32 || exact) return launch_lad_bwd_exact(p, dtype, dx, dz, s);
  if (p.grp == 1) return launch_walk_dims<uint16_t, 2, 2, lad::kDots>(p, dx, dz, s);
  return launch_walk_dims<uint16_t, 2, 2, lad::kParts>(p, dx, dz, s);
}

}  // namespace kda
