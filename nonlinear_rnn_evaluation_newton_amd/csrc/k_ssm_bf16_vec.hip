// Selective state space scan kernels, bf16 storage, vector access.
#include "k_ssm_impl.h"

namespace pr {
hipError_t launch_ssm_bf16_vec(const SsmArgs &a, int what, hipStream_t s) {
  return ssm_launch<uint16_t, true>(a, what, s);
}
}  // namespace pr
