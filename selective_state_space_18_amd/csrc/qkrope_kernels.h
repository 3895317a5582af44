// Norm of queries and keys over each head, with the position's rotation in the
// same pass (gfx950): forward and backward.
//
// Per token (position m) and head of D values, weight w (1 if null):
//   n = x * rstd * w,   rstd = 1 / sqrt(mean(x^2) + eps)
//   (y_a, y_b) = (n_a cos - n_b sin, n_a sin + n_b cos),  angle m * freqs[i]
// for the R/2 pairs i of the first R values, (i, i + R/2) or (2i, 2i + 1).
// Backward, with u = dy turned back, z = x * rstd and g = u * w:
//   dx = rstd (g - z mean(g z)),   dw = sum over tokens and heads of u z
//
// Work layout: a head is cut into units of two runs of kVec values: in halves,
// the runs i and i + R/2 that turn into each other, then the rest two by two;
// interleaved, neighbours.  A team of lanes holds one head, kUnits units a lane,
// so every value is read once and pairs never cross lanes.  A block takes a few
// tokens: their cosines and sines are computed once into LDS (in 64 bits, the
// angle reduced to its part of a turn, which keeps far positions exact) and
// serve all heads of q and k.
//
// What bounds it: HBM.  65536 tokens of 40 + 40 heads of 128, bf16: forward 470 us,
// 5.7 TB/s of reads and writes (a device copy: 4.9); 64 + 16 heads, interleaved: 505 us
// forward, 765 us backward (5.3 TB/s).  256 tokens of 64 + 64 heads take 12 us, trips of
// latency one after another: the angles, q's heads, k's; 4099 tokens of 7 + 1 heads of 96 in
// fp32 9 + 16 us and 5 for the sums.  Single values a lane are slower than the bytes: 65536
// tokens of 64 heads of 96 with 24 turned in halves 827 us, of 80 with 20 turned 802 us.
#pragma once

#include "attn_launch.h"
#include "ssm_device.h"

namespace ssm {

constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 2048;  // most pairs of a block's tokens

// kVec stored values.
template <typename T, int kVec>
struct RopeRun {
    T v[kVec];
};

// Sum over aligned teams of Q lanes, in every lane.
template <int Q>
__device__ __forceinline__ float rope_sum(float v) {
    v = lane_group_sum<(Q < 8 ? Q : 8)>(v);
#pragma unroll
    for (int o = 8; o < Q; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

// Where a unit's two runs lie, which of them exist, and its first pair.
struct RopeUnit {
    int a, b;    // first value of each run; >= D: none
    int pair;    // pair of value 0 (interleaved: pairs pair .. in both runs, one run after the other)
    bool turns;  // halves: the runs turn into each other
};
template <int kVec, bool kInter>
__device__ __forceinline__ RopeUnit rope_unit(int i, int D, int R) {
    RopeUnit u;
    if (kInter) {
        u.a = 2 * kVec * i, u.b = u.a + kVec;
        u.pair = kVec * i, u.turns = true;
    } else {
        const int half = R / 2, pairs = half / kVec;
        u.turns = i < pairs;
        u.a = u.turns ? kVec * i : R + 2 * kVec * (i - pairs);
        u.b = u.turns ? u.a + half : u.a + kVec;
        u.pair = u.turns ? kVec * i : 0;
    }
    if (u.a >= D) u.a = D;
    if (u.b >= D) u.b = D;
    return u;
}

// One head in the registers of its team.
template <typename T, int kVec, int kUnits, bool kInter>
struct RopeHead {
    RopeRun<T, kVec> r[kUnits][2];
    __device__ __forceinline__ void load(const T *x, const RopeUnit (&u)[kUnits], int D) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            if (u[k].a < D) r[k][0] = *reinterpret_cast<const RopeRun<T, kVec> *>(
                __builtin_assume_aligned(x + u[k].a, kVec * sizeof(T)));
            if (u[k].b < D) r[k][1] = *reinterpret_cast<const RopeRun<T, kVec> *>(
                __builtin_assume_aligned(x + u[k].b, kVec * sizeof(T)));
        }
    }
    __device__ __forceinline__ void values(float (&v)[kUnits][2][kVec], const RopeUnit (&u)[kUnits], int D) const {
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                v[k][0][e] = u[k].a < D ? to_f32(r[k][0].v[e]) : 0.f;
                v[k][1][e] = u[k].b < D ? to_f32(r[k][1].v[e]) : 0.f;
            }
    }
};
template <typename T, int kVec, int kUnits>
__device__ __forceinline__ void rope_store(T *y, const float (&v)[kUnits][2][kVec], const RopeUnit (&u)[kUnits], int D) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int at = s ? u[k].b : u[k].a;
            RopeRun<T, kVec> r;
#pragma unroll
            for (int e = 0; e < kVec; ++e) r.v[e] = from_acc<T>(v[k][s][e]);
            if (at < D)
                *reinterpret_cast<RopeRun<T, kVec> *>(__builtin_assume_aligned(y + at, kVec * sizeof(T))) = r;
        }
}

// v's pairs turned by the angles of one token: cs[i] = (cos, sin) of pair i.
// kBack: by the opposite angles.
template <int kVec, int kUnits, bool kInter, bool kBack>
__device__ __forceinline__ void rope_turn(float (&v)[kUnits][2][kVec], const float2 *cs, const RopeUnit (&u)[kUnits],
                                          int half) {
    auto turn = [](float &a, float &b, float2 f) {
        const float s = kBack ? -f.y : f.y, x = a;
        a = fma_(x, f.x, -(b * s));
        b = fma_(x, s, b * f.x);
    };
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        if constexpr (kInter && kVec > 1) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < kVec; e += 2) {
                    const int pair = u[k].pair + (s * kVec + e) / 2;
                    if (pair < half) turn(v[k][s][e], v[k][s][e + 1], cs[pair]);
                }
        } else if constexpr (kInter) {
            if (u[k].pair < half) turn(v[k][0][0], v[k][1][0], cs[u[k].pair]);
        } else {
            if (u[k].turns)
#pragma unroll
                for (int e = 0; e < kVec; ++e) turn(v[k][0][e], v[k][1][e], cs[u[k].pair + e]);
        }
    }
}

// Cosine and sine of `turns` (-1/2 to 1/2) of a full turn, each rounded once: the
// angle from the nearest quarter turn, its Taylor series in fp64 (the terms left out
// are below 2^-37 of 1, and of the sine), and the quarter turns by exchange and sign.
// (The library's fp64 function takes 20 registers more, and the backward a wave off every
// SIMD: 31.0 us for a training step of 4099 tokens of 8 heads, 29.1 this way.)
// kScalar, in the backward: the series' factors in scalar registers, where the compiler would
// keep them in 12 vector registers throughout the kernel (29.8 us).  The forward is slower
// with the fifth wave that this leaves room for: 65536 tokens of 80 heads 471 -> 479 us.
template <bool kScalar>
__device__ __forceinline__ float2 rope_cos_sin(double turns) {
    auto k = [](double v) {
        if (kScalar) __asm__ volatile("" : "+s"(v));
        return v;
    };
    const double quarters = rint(4.0 * turns), x = (turns - 0.25 * quarters) * k(6.283185307179586477), x2 = x * x;
    double s = fma_(x2, k(-1.0 / 39916800.0), k(1.0 / 362880.0)), c = fma_(x2, k(1.0 / 479001600.0), k(-1.0 / 3628800.0));
    s = fma_(x2, s, k(-1.0 / 5040.0)), c = fma_(x2, c, k(1.0 / 40320.0));
    s = fma_(x2, s, k(1.0 / 120.0)), c = fma_(x2, c, k(-1.0 / 720.0));
    s = fma_(x2, s, k(-1.0 / 6.0)), c = fma_(x2, c, k(1.0 / 24.0));
    c = fma_(x2, c, -0.5);
    const float sine = (float)fma_(x * x2, s, x), cosine = (float)fma_(x2, c, 1.0);
    const int n = (int)quarters;
    const float a = n & 1 ? sine : cosine, b = n & 1 ? cosine : sine;
    // by quarters: (c, s), (-s, c), (-c, -s), (s, -c)
    return make_float2((n + 1) & 2 ? -a : a, n & 2 ? -b : b);
}

// The cosines and sines of `tokens` tokens from `first` on.
template <bool kBwd>
__device__ __forceinline__ void rope_table(float2 *cs, const RopeParams &p, int64_t first, int tokens, int half) {
    for (int i = threadIdx.x; i < tokens * half; i += kRopeThreads) {
        const int t = i / half;
        constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
        const double z = (double)p.positions[first + t] * (double)p.freqs[i - t * half] * kTurn;
        cs[i] = rope_cos_sin<kBwd>(z - rint(z));
    }
}

// kBwd: x and the gradient of y are read, dx is written, and the block's sums
// of dweight leave as row blockIdx.x of p.part.
template <typename T, int kVec, int kTeam, int kUnits, bool kInter, bool kBwd>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeParams p) {
    constexpr int kTeams = kRopeThreads / kTeam;
    __shared__ __attribute__((aligned(16))) float2 cs[kRopeTable];
    const int lane = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
    const int half = p.R / 2;
    const float inv = 1.0f / (float)p.D;
    RopeUnit u[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) u[k] = rope_unit<kVec, kInter>(lane + k * kTeam, p.D, p.R);
    float dw[2][kBwd ? kUnits : 1][2][kVec];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < (kBwd ? kUnits : 1); ++k)
#pragma unroll
            for (int e = 0; e < kVec; ++e) dw[w][k][0][e] = dw[w][k][1][e] = 0.f;

    const int64_t batches = (p.rows + p.tokens - 1) / p.tokens;
    for (int64_t batch = blockIdx.x; batch < batches; batch += gridDim.x) {
        const int64_t first = batch * p.tokens;
        const int tokens = (int)(p.rows - first < p.tokens ? p.rows - first : p.tokens);
        if (batch != (int64_t)blockIdx.x) __syncthreads();  // the last tokens' angles are read
        rope_table<kBwd>(cs, p, first, tokens, half);
        __syncthreads();
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int H = which ? p.Hk : p.Hq;
            // this block's heads
            const int h0 = (int)((int64_t)H * blockIdx.y / gridDim.y), h1 = (int)((int64_t)H * (blockIdx.y + 1) / gridDim.y);
            const int heads = h1 - h0, items = tokens * heads;
            const T *x = static_cast<const T *>(which ? p.k : p.q) + first * H * p.D;
            const T *d = static_cast<const T *>(which ? p.dk : p.dq) + (kBwd ? first * H * p.D : 0);
            T *y = static_cast<T *>(which ? p.k_out : p.q_out) + first * H * p.D;
            const float *weight = which ? p.k_weight : p.q_weight;
            float w[kUnits][2][kVec];
#pragma unroll
            for (int k = 0; k < kUnits; ++k)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    w[k][0][e] = weight && u[k].a < p.D ? weight[u[k].a + e] : 1.f;
                    w[k][1][e] = weight && u[k].b < p.D ? weight[u[k].b + e] : 1.f;
                }
            auto at = [&](int item, int &token) {
                token = item / heads;
                return ((int64_t)token * H + h0 + (item - token * heads)) * p.D;
            };
            RopeHead<T, kVec, kUnits, kInter> nx, nd;
            int token = 0, next_token = 0;
            int64_t here = 0, next = 0;
            if (team < items) {
                next = at(team, next_token);
                nx.load(x + next, u, p.D);
                if (kBwd) nd.load(d + next, u, p.D);
            }
            for (int item = team; item < items; item += kTeams) {
                float v[kUnits][2][kVec], g[kUnits][2][kVec];
                nx.values(v, u, p.D);
                if (kBwd) nd.values(g, u, p.D);
                here = next, token = next_token;
                if (item + kTeams < items) {  // the next head's values on their way
                    next = at(item + kTeams, next_token);
                    nx.load(x + next, u, p.D);
                    if (kBwd) nd.load(d + next, u, p.D);
                }
                float sq = 0.f, gx = 0.f;
#pragma unroll
                for (int k = 0; k < kUnits; ++k)
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        sq = fma_(v[k][1][e], v[k][1][e], fma_(v[k][0][e], v[k][0][e], sq));
                const float rstd = 1.0f / sqrtf(fma_(rope_sum<kTeam>(sq), inv, p.eps));
                if constexpr (!kBwd) {
#pragma unroll
                    for (int k = 0; k < kUnits; ++k)
#pragma unroll
                        for (int e = 0; e < kVec; ++e) {
                            v[k][0][e] *= rstd * w[k][0][e];
                            v[k][1][e] *= rstd * w[k][1][e];
                        }
                    rope_turn<kVec, kUnits, kInter, false>(v, cs + token * half, u, half);
                    rope_store<T, kVec, kUnits>(y + here, v, u, p.D);
                } else {
                    rope_turn<kVec, kUnits, kInter, true>(g, cs + token * half, u, half);
#pragma unroll
                    for (int k = 0; k < kUnits; ++k)
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int e = 0; e < kVec; ++e) {
                                v[k][s][e] *= rstd;
                                dw[which][k][s][e] = fma_(g[k][s][e], v[k][s][e], dw[which][k][s][e]);
                                g[k][s][e] *= w[k][s][e];
                                gx = fma_(g[k][s][e], v[k][s][e], gx);
                            }
                    const float mean = rope_sum<kTeam>(gx) * inv;
#pragma unroll
                    for (int k = 0; k < kUnits; ++k)
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int e = 0; e < kVec; ++e) v[k][s][e] = rstd * fma_(-v[k][s][e], mean, g[k][s][e]);
                    rope_store<T, kVec, kUnits>(y + here, v, u, p.D);
                }
            }
        }
    }
    if constexpr (kBwd) {
        if (p.part == nullptr) return;
        // the teams' sums of one weight at a time, joined in the order of the teams
        __shared__ float sums[kRopeThreads * kUnits * 2 * kVec];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kUnits; ++k)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    float *to = sums + ((team * kUnits + k) * 2 * kVec + e) * kTeam + lane;
                    to[0] = dw[w][k][0][e];
                    to[kVec * kTeam] = dw[w][k][1][e];
                }
            __syncthreads();
            if (team == 0) {
                float *to = p.part + ((int64_t)blockIdx.x * 2 + w) * p.D;
#pragma unroll
                for (int k = 0; k < kUnits; ++k)
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int e = 0; e < kVec; ++e) {
                            float v = 0.f;
                            for (int t = 0; t < kTeams; ++t)
                                v += sums[((t * kUnits + k) * 2 * kVec + s * kVec + e) * kTeam + lane];
                            const int at = s ? u[k].b : u[k].a;
                            if (at < p.D) to[at + e] = v;
                        }
            }
        }
    }
}

template <int N>
struct RopeInt {
    static constexpr int value = N;
};

// Calls f(values a run, lanes a head, units a lane) with the shape for heads of
// D values: 16-byte runs where no run or pair is cut and every address allows
// it (bf16 heads of 128: 8 lanes), else single values, a wave to a head.
template <typename T, typename F>
void rope_shape(const RopeParams &p, F f) {
    constexpr int W = 16 / (int)sizeof(T);
    const void *ptrs[] = {p.q, p.k, p.dq, p.dk, p.q_out, p.k_out};
    uintptr_t bits = 0;
    for (const void *q : ptrs) bits |= (uintptr_t)q;
    const bool whole = p.D % W == 0 && bits % 16 == 0 && (p.interleaved || p.R % (2 * W) == 0);
    const int units = p.interleaved ? (p.D / W + 1) / 2 : p.R / (2 * W) + ((p.D - p.R) / W + 1) / 2;
    if (whole && units <= 4) f(RopeInt<W>(), RopeInt<4>(), RopeInt<1>());
    else if (whole && units <= 8) f(RopeInt<W>(), RopeInt<8>(), RopeInt<1>());
    else if (whole && units <= 16) f(RopeInt<W>(), RopeInt<16>(), RopeInt<1>());
    else if (whole && units <= 64) f(RopeInt<W>(), RopeInt<64>(), RopeInt<1>());
    else if (p.D <= 128) f(RopeInt<1>(), RopeInt<64>(), RopeInt<1>());
    else if (p.D <= 256) f(RopeInt<1>(), RopeInt<64>(), RopeInt<2>());
    else f(RopeInt<1>(), RopeInt<64>(), RopeInt<kRopeMaxHead / 128>());
}

// Tokens of a block and blocks of the grid.  Many tokens a block when there are
// many (the angles' table and the weights are then set up once for more heads), a part of
// a token's heads each when there are few.
struct RopeGrid {
    int tokens;
    int64_t x;
    unsigned y;
};
inline RopeGrid rope_grid(const RopeParams &p, int teams, bool bwd) {
    RopeGrid g;
    const int heads = p.Hq + p.Hk, half = p.R / 2 > 0 ? p.R / 2 : 1;
    const int64_t cus = p.cus > 0 ? p.cus : 256;
    int64_t tokens = (8 * teams + heads - 1) / heads;  // about 8 heads a team
    if (tokens > kRopeTable / half) tokens = kRopeTable / half;
    if (tokens > p.rows / (4 * cus)) tokens = p.rows / (4 * cus);
    if (tokens < 1) tokens = 1;
    g.tokens = (int)tokens;
    g.x = (p.rows + tokens - 1) / tokens;
    const int64_t passes = (heads + teams - 1) / teams, want = 4 * cus / g.x;
    g.y = bwd ? 1u : (unsigned)(want < 1 ? 1 : want < passes ? want : passes);
    if (bwd) {
        // blocks stay for many tokens and sum dweight in registers, in chains of
        // 256 heads at most
        const int64_t chain = (p.rows * heads + teams * 256 - 1) / (teams * 256);
        const int64_t most = chain > 8 * cus ? chain : 8 * cus;
        if (g.x > most) g.x = most;
    }
    if (g.x > (1 << 22)) g.x = 1 << 22;  // (blocks walk on by the grid)
    return g;
}

template <typename T>
hipError_t rope_t(RopePass pass, RopeParams &p, size_t *bytes, hipStream_t s) {
    hipError_t e = hipSuccess;
    rope_shape<T>(p, [&](auto vec, auto team, auto units) {
        constexpr int kVec = decltype(vec)::value, kTeam = decltype(team)::value, kUnits = decltype(units)::value;
        const bool bwd = pass != RopePass::kForward;
        const RopeGrid g = rope_grid(p, kRopeThreads / kTeam, bwd);
        p.tokens = g.tokens;
        const dim3 grid((unsigned)g.x, g.y), block(kRopeThreads);
        if (pass == RopePass::kPlan) {
            *bytes = (size_t)g.x * 2 * (size_t)p.D * 4;
        } else if (pass == RopePass::kReduce) {
            e = rope_reduce(p, g.x, s);
        } else if (pass == RopePass::kForward) {
            if (p.interleaved)
                hipLaunchKernelGGL((rope_kernel<T, kVec, kTeam, kUnits, true, false>), grid, block, 0, s, p);
            else
                hipLaunchKernelGGL((rope_kernel<T, kVec, kTeam, kUnits, false, false>), grid, block, 0, s, p);
        } else {
            if (p.interleaved)
                hipLaunchKernelGGL((rope_kernel<T, kVec, kTeam, kUnits, true, true>), grid, block, 0, s, p);
            else
                hipLaunchKernelGGL((rope_kernel<T, kVec, kTeam, kUnits, false, true>), grid, block, 0, s, p);
        }
    });
    return e != hipSuccess ? e : hipGetLastError();
}

}  // namespace ssm
