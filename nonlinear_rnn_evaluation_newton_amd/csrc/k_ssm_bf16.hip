// Selective state space scan kernels, bf16 storage, element access.
#include "k_ssm_impl.h"

namespace pr {
hipError_t launch_ssm_bf16(const SsmArgs &a, int what, hipStream_t s) {
  return ssm_launch<uint16_t, false>(a, what, s);
}
}  // namespace pr
