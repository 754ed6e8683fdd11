// Selective state space scan kernels, bf16 storage.
#include "k_ssm_impl.h"

namespace pr {
hipError_t launch_ssm_bf16(const SsmArgs &a, int what, hipStream_t s) { return ssm_launch<uint16_t>(a, what, s); }
}  // namespace pr
