// Layer norm (gfx950): forward with an optional residual add, backward with
// the reduction of the weight's and bias's gradients.
//
// Rows of Dm channels in groups of P; per group, with s = x (+ residual,
// rounded to the storage type):
//   mean = sum s / P,  rstd = 1 / sqrt(sum (s - mean)^2 / P + eps)
//   y = (s - mean) rstd weight + bias
// Backward, z = (s - mean) rstd and q = dy weight:
//   ds = rstd (q - mean(q) - z mean(q z)) (+ dsum)
//   dweight = sum over rows of dy z,  dbias = sum over rows of dy
// All arithmetic and sums are fp32; the variance is summed from the centred
// values, so an offset common to a group costs no accuracy.
#pragma once

#include "ssm_device.h"
#include "ssm_launch.h"

namespace ssm {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// One wave per (row, group).
template <typename T>
__global__ __launch_bounds__(64) void norm_fwd_kernel(NormParams p) {
    const int64_t ng = p.Dm / p.group;
    const int64_t row = blockIdx.x / ng, gr = blockIdx.x % ng;
    const int64_t base = row * p.Dm + gr * p.group;
    const T *x = static_cast<const T *>(p.x) + base;
    const T *res = p.residual ? static_cast<const T *>(p.residual) + base : nullptr;
    T *sum = p.sum ? static_cast<T *>(p.sum) + base : nullptr;
    T *y = static_cast<T *>(p.y) + base;
    const int P = (int)p.group, lane = threadIdx.x;
    auto value = [&](int c) {
        const float v = to_f32(x[c]);
        return res ? to_f32(from_acc<T>(v + to_f32(res[c]))) : v;
    };
    float a = 0.f;
    for (int c = lane; c < P; c += 64) a += value(c);
    const float mean = wave_sum(a) / (float)P;
    float b = 0.f;
    for (int c = lane; c < P; c += 64) {
        const float v = value(c) - mean;
        b += v * v;
    }
    const float rstd = 1.0f / sqrtf(wave_sum(b) / (float)P + p.eps);
    for (int c = lane; c < P; c += 64) {
        const float v = value(c);
        const float w = p.weight ? p.weight[gr * p.group + c] : 1.f;
        const float o = p.bias ? p.bias[gr * p.group + c] : 0.f;
        y[c] = from_acc<T>((v - mean) * rstd * w + o);
        if (sum) sum[c] = from_acc<T>(v);
    }
    if (lane == 0) {
        if (p.mean) p.mean[blockIdx.x] = mean;
        if (p.rstd) p.rstd[blockIdx.x] = rstd;
    }
}

template <typename T>
__global__ __launch_bounds__(64) void norm_bwd_kernel(NormBwdParams p) {
    const int64_t ng = p.Dm / p.group;
    const int64_t row = blockIdx.x / ng, gr = blockIdx.x % ng;
    const int64_t base = row * p.Dm + gr * p.group;
    const T *s = static_cast<const T *>(p.s) + base, *dy = static_cast<const T *>(p.dy) + base;
    const T *dsum = p.dsum ? static_cast<const T *>(p.dsum) + base : nullptr;
    T *dx = static_cast<T *>(p.dx) + base;
    const float *w = p.weight ? p.weight + gr * p.group : nullptr;
    const int P = (int)p.group, lane = threadIdx.x;
    const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x];
    float a = 0.f, b = 0.f;
    for (int c = lane; c < P; c += 64) {
        const float q = to_f32(dy[c]) * (w ? w[c] : 1.f);
        a += q;
        b += q * (to_f32(s[c]) - mean) * rstd;
    }
    a = wave_sum(a) / (float)P;
    b = wave_sum(b) / (float)P;
    for (int c = lane; c < P; c += 64) {
        const float q = to_f32(dy[c]) * (w ? w[c] : 1.f);
        const float z = (to_f32(s[c]) - mean) * rstd;
        dx[c] = from_acc<T>(rstd * (q - a - z * b) + (dsum ? to_f32(dsum[c]) : 0.f));
    }
}

// One thread per column.
template <typename T>
__global__ __launch_bounds__(64) void norm_bwd_reduce_kernel(NormBwdParams p) {
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (c >= p.Dm) return;
    const int64_t ng = p.Dm / p.group, gr = c / p.group;
    const T *s = static_cast<const T *>(p.s), *dy = static_cast<const T *>(p.dy);
    float dw = 0.f, db = 0.f;
    for (int64_t row = 0; row < p.rows; ++row) {
        const float v = to_f32(dy[row * p.Dm + c]);
        dw += v * (to_f32(s[row * p.Dm + c]) - p.mean[row * ng + gr]) * p.rstd[row * ng + gr];
        db += v;
    }
    if (p.dweight) p.dweight[c] = dw;
    if (p.dbias) p.dbias[c] = db;
}

template <typename T>
hipError_t norm_fwd_t(const NormParams &p, hipStream_t s) {
    hipLaunchKernelGGL(norm_fwd_kernel<T>, dim3((unsigned)(p.rows * (p.Dm / p.group))), dim3(64), 0, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t norm_bwd_t(const NormBwdParams &p, hipStream_t s) {
    hipLaunchKernelGGL(norm_bwd_kernel<T>, dim3((unsigned)(p.rows * (p.Dm / p.group))), dim3(64), 0, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t norm_bwd_reduce_t(const NormBwdParams &p, hipStream_t s) {
    hipLaunchKernelGGL(norm_bwd_reduce_kernel<T>, dim3((unsigned)((p.Dm + 63) / 64)), dim3(64), 0, s, p);
    return hipGetLastError();
}

}  // namespace ssm
