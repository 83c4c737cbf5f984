// The segments' own states, from zero.
#include "lad_walk.h"

namespace kda {

hipError_t launch_lad_states(const LadParams& p, int dtype, int dx, int dz, hipStream_t s) {
  return dtype == KDA_DTYPE_BF16 ? launch_walk_dims<uint16_t, 3, 2, lad::kStates>(p, dx, dz, s) : launch_walk_dims<float, 3, 2, lad::kStates>(p, dx, dz, s);
}

}  // namespace kda
