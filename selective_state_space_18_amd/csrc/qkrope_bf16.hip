// Norm and rotation of queries and keys, bf16 storage.
#include "qkrope_kernels.h"

namespace ssm {

hipError_t rope_bf16(RopePass pass, RopeParams &p, size_t *bytes, hipStream_t s) { return rope_t<bf16>(pass, p, bytes, s); }

}  // namespace ssm
