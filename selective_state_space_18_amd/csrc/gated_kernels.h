// Gated linear recurrence (gfx950): forward scan, backward, decode step.
//
// Per batch row and channel, with A <= 0 and the gates' raw inputs r, i:
//   s = sigmoid(r_t), g = sigmoid(i_t), u = A s, a = exp(u), m = sqrt(1 - a^2)
//   h_t = a h_{t-1} + m g x_t,   y_t = h_t
// Backward, lam_t = dL/dh_t:
//   lam_t = dy_t + a_{t+1} lam_{t+1}
//   dx = lam m g,  di = lam m x g (1 - g)
//   du = lam (a h_{t-1} - g x a^2 / m),  dr = du A s (1 - s),  dA = sum du s
// Where m = 0 (u = 0: A = 0, or the gate underflows) the quotient a^2/m is
// taken as 0: its product with A s has that limit, and for dA, whose
// derivative there is not finite, it is the convention.
//
// Arithmetic is fp32 for both storage types.  bf16 storage takes exp, sqrt
// and 1/x from the transcendental unit (each about one ulp of fp32); fp32
// storage takes the accurate library functions.
#pragma once

#include "ssm_device.h"
#include "ssm_launch.h"

namespace ssm {

// exp(-v) + 1 inverted: the logistic function.
template <typename T>
__device__ __forceinline__ float sigmoid_(float v) {
    if constexpr (sizeof(T) == 4)
        return 1.0f / (1.0f + expf(-v));
    else
        return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

// a = exp(u) and m = sqrt(1 - a^2) for u <= 0.  1 - a^2 cancels near u = 0;
// there it is 2 a sinh(v), v = -u, with the series v (1 + v^2/6 + v^4/120 +
// v^6/5040), whose truncation for v < 0.5 is below v^8/362880 = 1.1e-8.
template <typename T>
__device__ __forceinline__ void decay_(float u, float &a, float &m) {
    if constexpr (sizeof(T) == 4) {
        a = expf(u);
        m = sqrtf(-expm1f(2.0f * u));
    } else {
        a = fast_exp2(u * kLog2e);
        const float v2 = u * u;
        const float p = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(v2, 1.0f / 5040.0f, 1.0f / 120.0f), v2, 1.0f / 6.0f),
                                       v2, 1.0f);
        const float near = -2.0f * u * a * p;
        const float far = __builtin_fmaf(-a, a, 1.0f);
        m = __builtin_amdgcn_sqrtf(u > -0.5f ? near : far);
    }
}

// ---------------------------------------------------------------------------
// One thread per channel, one step after another.

template <typename T>
__global__ __launch_bounds__(64) void gated_fwd_kernel(GatedParams p) {
    const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (d >= p.Dm) return;
    const float A = p.A[d];
    const T *x = static_cast<const T *>(p.x), *r = static_cast<const T *>(p.r), *gi = static_cast<const T *>(p.i);
    T *y = static_cast<T *>(p.y);
    const bool packed = p.cu != nullptr;
    int64_t k = packed ? -1 : b;
    float h = packed ? 0.f : (p.h_init ? p.h_init[b * p.Dm + d] : 0.f);
    const int64_t tiles = (p.L + kGatedCarrySteps - 1) / kGatedCarrySteps;
    for (int64_t t = 0; t < p.L; ++t) {
        if (p.carry && t % kGatedCarrySteps == 0) p.carry[(b * tiles + t / kGatedCarrySteps) * p.Dm + d] = h;
        if (packed && k < p.nseq - 1 && p.cu[k + 1] <= t) {
            if (k >= 0 && p.h_final) p.h_final[k * p.Dm + d] = h;
            while (k < p.nseq - 1 && p.cu[k + 1] <= t) ++k;
            h = p.h_init ? p.h_init[k * p.Dm + d] : 0.f;
        }
        const int64_t at = (b * p.L + t) * p.Dm + d;
        float a, m;
        decay_<T>(A * sigmoid_<T>(to_f32(r[at])), a, m);
        h = __builtin_fmaf(a, h, m * sigmoid_<T>(to_f32(gi[at])) * to_f32(x[at]));
        if (y) y[at] = from_acc<T>(h);
    }
    if (p.h_final && k >= 0) p.h_final[k * p.Dm + d] = h;
}

template <typename T>
__global__ __launch_bounds__(64) void gated_bwd_kernel(GatedBwdParams q) {
    const GatedParams &p = q.f;
    const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (d >= p.Dm) return;
    const float A = p.A[d];
    const T *x = static_cast<const T *>(p.x), *r = static_cast<const T *>(p.r), *gi = static_cast<const T *>(p.i);
    const T *dy = static_cast<const T *>(q.dy);
    T *dx = static_cast<T *>(q.dx), *dr = static_cast<T *>(q.dr), *di = static_cast<T *>(q.di);
    const bool packed = p.cu != nullptr;
    const int64_t tiles = (p.L + kGatedCarrySteps - 1) / kGatedCarrySteps;
    float dA = 0.f;
    for (int64_t b = 0; b < p.Bsz; ++b) {
        int64_t k = b;  // the sequence the current step belongs to
        if (packed) {
            k = p.nseq - 1;
            while (k > 0 && p.cu[k] >= p.L) --k;
        }
        float e = q.dh_final ? q.dh_final[k * p.Dm + d] : 0.f;
        for (int64_t t = p.L - 1; t >= 0; --t) {
            // the state before step t, from the carry of its tile
            const int64_t t0 = t / kGatedCarrySteps * kGatedCarrySteps;
            const bool start = packed ? p.cu[k] == t : false;
            float h = p.carry[(b * tiles + t0 / kGatedCarrySteps) * p.Dm + d];
            int64_t from = t0;
            if (packed && p.cu[k] >= t0) {
                from = p.cu[k];
                h = p.h_init ? p.h_init[k * p.Dm + d] : 0.f;
            }
            for (int64_t c = from; c < t; ++c) {
                const int64_t at = (b * p.L + c) * p.Dm + d;
                float a, m;
                decay_<T>(A * sigmoid_<T>(to_f32(r[at])), a, m);
                h = __builtin_fmaf(a, h, m * sigmoid_<T>(to_f32(gi[at])) * to_f32(x[at]));
            }
            const int64_t at = (b * p.L + t) * p.Dm + d;
            const float s = sigmoid_<T>(to_f32(r[at])), g = sigmoid_<T>(to_f32(gi[at])), xv = to_f32(x[at]);
            float a, m;
            decay_<T>(A * s, a, m);
            const float lam = to_f32(dy[at]) + e;
            const float lm = lam * m * g;
            const float quot = m > 0.f ? g * xv * a * a / m : 0.f;
            const float du = lam * (a * h - quot);
            dx[at] = from_acc<T>(lm);
            di[at] = from_acc<T>(lm * xv * (1.f - g));
            dr[at] = from_acc<T>(du * A * s * (1.f - s));
            dA += du * s;
            e = a * lam;
            if (start) {
                if (q.dh_init) q.dh_init[k * p.Dm + d] = e;
                if (t > 0) {
                    while (k > 0 && p.cu[k] >= t) --k;
                    e = q.dh_final ? q.dh_final[k * p.Dm + d] : 0.f;
                }
            }
        }
        if (!packed && q.dh_init) q.dh_init[b * p.Dm + d] = e;
    }
    q.dA[d] = dA;
}

template <typename T>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedStepParams p) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= p.Bsz * p.Dm) return;
    const float A = p.A[at % p.Dm];
    float a, m;
    decay_<T>(A * sigmoid_<T>(to_f32(static_cast<const T *>(p.r)[at])), a, m);
    const float in = m * sigmoid_<T>(to_f32(static_cast<const T *>(p.i)[at])) * to_f32(static_cast<const T *>(p.x)[at]);
    const float h = __builtin_fmaf(a, p.h[at], in);
    p.h_out[at] = h;
    static_cast<T *>(p.y)[at] = from_acc<T>(h);
}

template <typename T>
hipError_t gated_fwd_t(const GatedParams &p, hipStream_t s) {
    const dim3 grid((unsigned)((p.Dm + 63) / 64), (unsigned)p.Bsz);
    hipLaunchKernelGGL(gated_fwd_kernel<T>, grid, dim3(64), 0, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t gated_bwd_t(const GatedBwdParams &q, hipStream_t s) {
    hipLaunchKernelGGL(gated_bwd_kernel<T>, dim3((unsigned)((q.f.Dm + 63) / 64)), dim3(64), 0, s, q);
    return hipGetLastError();
}

template <typename T>
hipError_t gated_step_t(const GatedStepParams &p, hipStream_t s) {
    hipLaunchKernelGGL(gated_step_kernel<T>, dim3((unsigned)((p.Bsz * p.Dm + 255) / 256)), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace ssm
