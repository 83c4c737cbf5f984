// The gradients of q, k and v: the walk over other tensors, its states only entering results of the inputs' type.
#include "lad_walk.h"

namespace kda {

hipError_t launch_lad_bwd(const LadParams& p, int dtype, int dx, int dz, hipStream_t s) {
  return dtype == KDA_DTYPE_BF16 ? launch_walk_dims<uint16_t, 2, true>(p, dx, dz, s) : launch_walk_dims<float, 2, true>(p, dx, dz, s);
}

}  // namespace kda
