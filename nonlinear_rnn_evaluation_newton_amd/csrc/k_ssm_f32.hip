// Selective state space scan kernels, fp32 storage, element access.
#include "k_ssm_impl.h"

namespace pr {
hipError_t launch_ssm_f32(const SsmArgs &a, int what, hipStream_t s) {
  return ssm_launch<float, false>(a, what, s);
}
}  // namespace pr
