// Norm and rotation of queries and keys, fp32 storage, and the sums of dweight.
#include "qkrope_kernels.h"

namespace ssm {

namespace {

// dst[w][d] = sum over blocks of part[block][w][d]: 16 chains of blocks a
// column, joined in their order.
__global__ __launch_bounds__(1024) void rope_reduce_kernel(const float *part, int64_t blocks, int D, float *dq_weight,
                                                           float *dk_weight) {
    __shared__ float sums[16][kWave];
    float *dst = blockIdx.y ? dk_weight : dq_weight;
    if (dst == nullptr) return;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int d = (int)blockIdx.x * kWave + lane;
    const float *src = part + (int64_t)blockIdx.y * D + d;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (d < D)
        for (int64_t b = wave; b < blocks; b += 64)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (b + 16 * k < blocks) v[k] += src[(b + 16 * k) * 2 * D];
    sums[wave][lane] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (wave == 0 && d < D) {
        float all = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) all += sums[w][lane];
        dst[d] = all;
    }
}

}  // namespace

hipError_t rope_reduce(const RopeParams &p, int64_t blocks, hipStream_t s) {
    hipLaunchKernelGGL(rope_reduce_kernel, dim3((unsigned)((p.D + kWave - 1) / kWave), 2), dim3(1024), 0, s, p.part, blocks,
                       p.D, p.dq_weight, p.dk_weight);
    return hipGetLastError();
}

hipError_t rope_f32(RopePass pass, RopeParams &p, size_t *bytes, hipStream_t s) { return rope_t<float>(pass, p, bytes, s); }

}  // namespace ssm
