// Gated linear recurrence, fp32 storage.
#include "gated_kernels.h"

namespace ssm {

hipError_t gated_fwd_f32(const GatedParams &p, hipStream_t s) { return gated_fwd_t<float>(p, s); }
hipError_t gated_bwd_f32(const GatedBwdParams &q, hipStream_t s) { return gated_bwd_t<float>(q, s); }
hipError_t gated_step_f32(const GatedStepParams &p, hipStream_t s) { return gated_step_t<float>(p, s); }

}  // namespace ssm
