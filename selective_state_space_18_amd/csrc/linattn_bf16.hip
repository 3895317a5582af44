// Linear attention, bf16 storage.
#include "linattn_kernels.h"

namespace ssm {

hipError_t lin_fit_bf16(int64_t nk, int64_t nv, int *blocks) { return lin_fit_t<bf16>(nk, nv, blocks); }
hipError_t lin_pass_bf16(LinPass pass, const LinParams &p, hipStream_t s) { return lin_pass_t<bf16>(pass, p, s); }
hipError_t lin_step_bf16(const LinStepParams &p, hipStream_t s) { return lin_step_t<bf16>(p, s); }

}  // namespace ssm
