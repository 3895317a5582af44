// Gated linear recurrence, fp32 storage.
#include "gated_kernels.h"

namespace ssm {

hipError_t gated_fwd_f32(GatedPass pass, GatedParams &p, void *scratch, GatedPlan *plan, hipStream_t s) {
    return gated_fwd_t<float>(pass, p, scratch, plan, s);
}
hipError_t gated_bwd_f32(GatedPass pass, GatedBwdParams &q, void *scratch, GatedPlan *plan, hipStream_t s) {
    return gated_bwd_t<float>(pass, q, scratch, plan, s);
}
hipError_t gated_step_f32(const GatedStepParams &p, hipStream_t s) { return gated_step_t<float>(p, s); }
hipError_t gated_states(const int64_t *cu, int64_t rows, const float *from, float *to, int64_t Dm, hipStream_t s) {
    return gated_states_launch(cu, rows, from, to, Dm, s);
}

}  // namespace ssm
