// Gated linear recurrence, bf16 storage.
#include "gated_kernels.h"

namespace ssm {

hipError_t gated_fwd_bf16(const GatedParams &p, hipStream_t s) { return gated_fwd_t<bf16>(p, s); }
hipError_t gated_bwd_bf16(const GatedBwdParams &q, hipStream_t s) { return gated_bwd_t<bf16>(q, s); }
hipError_t gated_step_bf16(const GatedStepParams &p, hipStream_t s) { return gated_step_t<bf16>(p, s); }

}  // namespace ssm
