// Selective state space scan kernels, fp32 storage, vector access.
#include "k_ssm_impl.h"

namespace pr {
hipError_t launch_ssm_f32_vec(const SsmArgs &a, int what, hipStream_t s) {
  return ssm_launch<float, true>(a, what, s);
}
}  // namespace pr
