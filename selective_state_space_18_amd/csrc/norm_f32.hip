// Layer norm, fp32 storage.
#include "norm_kernels.h"

namespace ssm {

hipError_t norm_fwd_f32(const NormParams &p, hipStream_t s) { return norm_fwd_t<float>(p, s); }
hipError_t norm_bwd_f32(NormPass pass, NormBwdParams &p, size_t *bytes, hipStream_t s) {
    return norm_bwd_t<float>(pass, p, bytes, s);
}

}  // namespace ssm
