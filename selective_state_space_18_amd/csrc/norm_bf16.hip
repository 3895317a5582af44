// Layer norm, bf16 storage.
#include "norm_kernels.h"

namespace ssm {

hipError_t norm_fwd_bf16(const NormParams &p, hipStream_t s) { return norm_fwd_t<bf16>(p, s); }
hipError_t norm_bwd_bf16(NormPass pass, NormBwdParams &p, size_t *bytes, hipStream_t s) {
    return norm_bwd_t<bf16>(pass, p, bytes, s);
}

}  // namespace ssm
