// Norm and rotation of queries and keys, fp32 storage, and the sums of dweight.
#include "qkrope_kernels.h"

namespace ssm {

namespace {

// dst[w][d] = sum over blocks of part[block][w][d].  A block takes 8 columns:
// 128 chains of rows a column, 8 loads of each in flight, joined pair by pair: one after
// another, the rounding of 128 adds would be most of the sums' error (2.9 in place of 0.6 units of 2^-24).  (Bound by
// the loads' latency: 2048 rows of two weights of 128 take 11 us, with 16 columns and 64
// chains 19, with 64 columns, 16 chains and 4 in flight 57.)
constexpr int kReduceCols = 8, kReduceChains = 128, kReduceAhead = 8;
__global__ __launch_bounds__(kReduceCols * kReduceChains) void rope_reduce_kernel(const float *part, int64_t blocks, int D,
                                                                                 float *dq_weight, float *dk_weight) {
    __shared__ float sums[kReduceChains][kReduceCols];
    float *dst = blockIdx.y ? dk_weight : dq_weight;
    if (dst == nullptr) return;
    const int col = threadIdx.x % kReduceCols, chain = threadIdx.x / kReduceCols;
    const int d = (int)blockIdx.x * kReduceCols + col;
    const float *src = part + (int64_t)blockIdx.y * D + d;
    float v[kReduceAhead] = {};
    if (d < D)
        for (int64_t b = chain; b < blocks; b += kReduceChains * kReduceAhead)
#pragma unroll
            for (int k = 0; k < kReduceAhead; ++k)
                if (b + kReduceChains * k < blocks) v[k] += src[(b + kReduceChains * k) * 2 * D];
#pragma unroll
    for (int o = 1; o < kReduceAhead; o <<= 1)
#pragma unroll
        for (int k = 0; k < kReduceAhead; k += 2 * o) v[k] += v[k + o];
    sums[chain][col] = v[0];
#pragma unroll
    for (int o = kReduceChains / 2; o > 0; o /= 2) {
        __syncthreads();
        if (chain < o) sums[chain][col] += sums[chain + o][col];
    }
    if (chain == 0 && d < D) dst[d] = sums[0][col];
}

}  // namespace

hipError_t rope_reduce(const RopeParams &p, int64_t blocks, hipStream_t s) {
    hipLaunchKernelGGL(rope_reduce_kernel, dim3((unsigned)((p.D + kReduceCols - 1) / kReduceCols), 2),
                       dim3(kReduceCols * kReduceChains), 0, s, p.part, blocks, p.D, p.dq_weight, p.dk_weight);
    return hipGetLastError();
}

hipError_t rope_f32(RopePass pass, RopeParams &p, size_t *bytes, hipStream_t s) { return rope_t<float>(pass, p, bytes, s); }

}  // namespace ssm
