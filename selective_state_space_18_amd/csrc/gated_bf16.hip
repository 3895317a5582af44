// Gated linear recurrence, bf16 storage.
#include "gated_kernels.h"

namespace ssm {

hipError_t gated_fwd_bf16(GatedPass pass, GatedParams &p, void *scratch, GatedPlan *plan, hipStream_t s) {
    return gated_fwd_t<bf16>(pass, p, scratch, plan, s);
}
hipError_t gated_bwd_bf16(GatedPass pass, GatedBwdParams &q, void *scratch, GatedPlan *plan, hipStream_t s) {
    return gated_bwd_t<bf16>(pass, q, scratch, plan, s);
}
hipError_t gated_step_bf16(const GatedStepParams &p, hipStream_t s) { return gated_step_t<bf16>(p, s); }

}  // namespace ssm
