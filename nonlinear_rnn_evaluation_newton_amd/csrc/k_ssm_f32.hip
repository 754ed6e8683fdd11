// Selective state space scan kernels, fp32 storage.
#include "k_ssm_impl.h"

namespace pr {
hipError_t launch_ssm_f32(const SsmArgs &a, int what, hipStream_t s) { return ssm_launch<float>(a, what, s); }
}  // namespace pr
