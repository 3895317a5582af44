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
// All arithmetic and sums are fp32; the variance is summed from centred
// values, so an offset common to a group costs no more than the rounding of the
// group's mean.
//
// Work layout: a team of lanes (8 to 64, or a whole block) holds one group in
// registers, kNv vectors of kVec channels per lane, and reads it once.  A block
// of teams covers consecutive groups of a row and walks down the rows, so a
// lane keeps its channels: weight and bias are loaded once, and the backward
// sums dweight and dbias of its channels in registers, kNormSumRows rows at a
// time.
//
// What bounds it: HBM; counters show every value read and written once.  bf16,
// 65536 rows of 5120 with residual and sum: forward 0.54 ms (5.0 TB/s of 8 bytes
// a value), backward 0.49 ms (5.5 TB/s, with dsum); in heads of 64, forward only,
// 0.255 ms (5.3 TB/s of 4 bytes).  Small calls are bound by their launch and one
// trip of latency: 256 rows of 8192 5.8 us, fp32 4099 rows of 777 9.0 us forward
// and 13.7 + 3.8 backward.  Where rows are shorter than a block of teams, its other
// lanes idle: 65536 rows of 64 take 42 us forward, 12 times their bytes.
#pragma once

#include "layer_launch.h"
#include "ssm_device.h"

namespace ssm {

// Sum over aligned groups of Q lanes, in every lane of the group.
template <int Q>
__device__ __forceinline__ float lanes_sum(float v) {
    v = lane_group_sum<(Q < 8 ? Q : 8)>(v);
    if constexpr (Q >= 16)  // row mirror: the other half of 16 lanes
        v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, false));
    if constexpr (Q >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (Q >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

// Lane 0's value (the first 16 lanes hold the sum of the waves).
__device__ __forceinline__ float uniform_f(float v) { return __int_as_float(uniform(__float_as_int(v))); }

// kVec stored values.
template <typename T, int kVec>
struct Stored {
    T v[kVec];
};
typedef u32x4 u32x4_loose __attribute__((aligned(2)));  // gfx950 reads and writes 16 bytes at any address

// The first n of kVec (16 bytes) stored values at p; the others are 0.  Not
// kLoose: n is 0 or kVec and p is 16-byte aligned.
template <typename T, int kVec, bool kLoose>
__device__ __forceinline__ Stored<T, kVec> load_vec(const T *p, int n) {
    static_assert(kVec * sizeof(T) == 16, "16 bytes");
    Stored<T, kVec> r;
    u32x4 w = {0, 0, 0, 0};
    if (kLoose ? n == kVec : n > 0) {
        if constexpr (kLoose)
            w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_loose *>(p));
        else
            w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
    }
    __builtin_memcpy(&r, &w, 16);
    if (kLoose && n > 0 && n < kVec) {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < n) r.v[e] = p[e];
    }
    return r;
}
template <typename T, int kVec, bool kLoose>
__device__ __forceinline__ void store_vec(T *p, int n, const Stored<T, kVec> &r) {
    u32x4 w;
    __builtin_memcpy(&w, &r, 16);
    if (kLoose ? n == kVec : n > 0) {
        if constexpr (kLoose)
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4_loose *>(p));
        else
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(p));
    }
    if (kLoose && n > 0 && n < kVec) {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < n) p[e] = r.v[e];
    }
}

// The first n of kVec parameters at p, or `none` where there are none (one
// branch, so that their loads are in flight together).
template <int kVec>
__device__ __forceinline__ void load_params(const float *p, bool given, int n, float none, float (&w)[kVec]) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[e] = none;
    if (given && n == kVec) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) w[e] = p[e];
    } else if (given) {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < n) w[e] = p[e];
    }
}

// A lane's place: its group, its number in the team and whether it has a group.
// kTeam = 0: the block is one team, of blockDim.x lanes.
template <int kVec, int kTeam>
struct NormLane {
    int64_t group;
    int lane, team;
    bool on;
    __device__ NormLane(int64_t groups) {
        team = kTeam ? kTeam : (int)blockDim.x;
        group = kTeam ? (int64_t)blockIdx.x * (256 / (kTeam ? kTeam : 256)) + threadIdx.x / (kTeam ? kTeam : 1)
                      : (int64_t)blockIdx.x;
        lane = kTeam ? threadIdx.x % (kTeam ? kTeam : 1) : threadIdx.x;
        on = group < groups;
    }
    // first channel, inside the group, of the lane's k-th vector
    __device__ int at(int k) const { return (lane + k * team) * kVec; }
};

// Channels of a group of P that wave z of a block-wide team holds.
template <int kVec, int kNv>
__device__ __forceinline__ int wave_channels(int P, int z, int team) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        const int c = P - (k * team + z * kWave) * kVec;
        n += c < 0 ? 0 : c > kWave * kVec ? kWave * kVec : c;
    }
    return n;
}

constexpr int kNormMaxWaves = 16;

// Rows whose terms of dweight and dbias are added up in one chain; a block's
// chains are then added to its row of partial sums, so that the error of a sum
// over n rows grows with this and n / this, not with n.
constexpr int kNormSumRows = 256;

// The next row's values are loaded before this row's sums (where a lane holds
// few enough channels for the registers that takes), so that loads are in flight
// beside the reduction and the stores: forward + backward of 65536 x 5120 1.38 ->
// 1.16 ms.
template <typename T, int kVec, int kTeam, int kNv, bool kLoose>
__global__ __launch_bounds__(kTeam ? 256 : 1024) void norm_fwd_kernel(NormParams p) {
    constexpr int kLanes = kTeam ? kTeam : kWave;
    constexpr bool kAhead = kNv * kVec <= 8;
    __shared__ float red[2][kNormMaxWaves][2];
    const int64_t ng = p.Dm / p.group;
    const NormLane<kVec, kTeam> me(ng);
    const int P = (int)p.group, wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const float inv = 1.0f / (float)P;
    int n[kNv];  // channels of each vector inside the group
    auto has = [&](int k, int e) { return kLoose ? e < n[k] : n[k] > 0; };
    float w[kNv][kVec], o[kNv][kVec];
    Stored<T, kVec> s[kNv], r[kNv];
    const int64_t col = me.group * P;
    auto load = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            const int64_t at = row * p.Dm + col + me.at(k);
            s[k] = load_vec<T, kVec, kLoose>(static_cast<const T *>(p.x) + at, n[k]);
            if (p.residual) r[k] = load_vec<T, kVec, kLoose>(static_cast<const T *>(p.residual) + at, n[k]);
        }
    };
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        const int left = me.on ? P - me.at(k) : 0;
        n[k] = left < 0 ? 0 : left > kVec ? kVec : left;
    }
    if (kAhead) load(blockIdx.y);
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        load_params<kVec>(p.weight + col + me.at(k), p.weight != nullptr, n[k], 1.f, w[k]);
        load_params<kVec>(p.bias + col + me.at(k), p.bias != nullptr, n[k], 0.f, o[k]);
    }
    const int waves = blockDim.x / kWave;
    // values this wave holds; and, for the waves' sums, lane z those of wave z
    const float mine = kTeam ? 1.f : (float)wave_channels<kVec, kNv>(P, wave, me.team);
    const float of_lane = kTeam || lane >= waves ? 0.f : (float)wave_channels<kVec, kNv>(P, lane, me.team);
    int turn = 0;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const int64_t base = row * p.Dm + col;
        if (!kAhead) load(row);
        float v[kNv][kVec], sum = 0.f;
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            if (p.residual) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) s[k].v[e] = from_acc<T>(to_f32(s[k].v[e]) + to_f32(r[k].v[e]));
                if (p.sum) store_vec<T, kVec, kLoose>(static_cast<T *>(p.sum) + base + me.at(k), n[k], s[k]);
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                v[k][e] = to_f32(s[k].v[e]);
                sum += v[k][e];
            }
        }
        if (kAhead && row + gridDim.y < p.rows) load(row + gridDim.y);
        // mean and squared deviations of what this wave (or team) holds
        sum = lanes_sum<kLanes>(sum);
        float mean = kTeam ? sum * inv : mine > 0.f ? sum / mine : 0.f;
        float dev = 0.f;
#pragma unroll
        for (int k = 0; k < kNv; ++k)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float c = has(k, e) ? v[k][e] - mean : 0.f;
                dev = __builtin_fmaf(c, c, dev);
            }
        dev = lanes_sum<kLanes>(dev);
        if constexpr (kTeam == 0) {
            // the waves' means and deviations joined: with d = mean_w - mean,
            // the squared deviations from the mean of all are dev_w + n_w d^2
            if (waves > 1) {
                if (lane == 0) {
                    red[turn][wave][0] = mean;
                    red[turn][wave][1] = dev;
                }
                __syncthreads();
                const float mw = lane < waves ? red[turn][lane % kNormMaxWaves][0] : 0.f;
                const float dw = lane < waves ? red[turn][lane % kNormMaxWaves][1] : 0.f;
                mean = uniform_f(lanes_sum<kNormMaxWaves>(of_lane * mw)) * inv;
                const float d = mw - mean;
                dev = uniform_f(lanes_sum<kNormMaxWaves>(__builtin_fmaf(of_lane * d, d, dw)));
                turn ^= 1;  // the next row's values go to the other buffer
            }
        }
        const float rstd = 1.0f / sqrtf(__builtin_fmaf(dev, inv, p.eps));
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            Stored<T, kVec> y;
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                y.v[e] = from_acc<T>(__builtin_fmaf((v[k][e] - mean) * rstd, w[k][e], o[k][e]));
            store_vec<T, kVec, kLoose>(static_cast<T *>(p.y) + base + me.at(k), n[k], y);
        }
        if (me.on && me.lane == 0) {
            if (p.mean) p.mean[row * ng + me.group] = mean;
            if (p.rstd) p.rstd[row * ng + me.group] = rstd;
        }
    }
}

template <typename T, int kVec, int kTeam, int kNv, bool kLoose>
__global__ __launch_bounds__(kTeam ? 256 : 1024) void norm_bwd_kernel(NormBwdParams p) {
    constexpr int kLanes = kTeam ? kTeam : kWave;
    constexpr bool kAhead = kNv * kVec <= 8;
    __shared__ float red[2][kNormMaxWaves][2];
    const int64_t ng = p.Dm / p.group;
    const NormLane<kVec, kTeam> me(ng);
    const int P = (int)p.group, wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const float inv = 1.0f / (float)P;
    int n[kNv];  // channels of each vector inside the group
    auto has = [&](int k, int e) { return kLoose ? e < n[k] : n[k] > 0; };
    float w[kNv][kVec], dw[kNv][kVec], db[kNv][kVec];
    Stored<T, kVec> s[kNv], g[kNv], r[kNv];
    float mean = 0.f, rstd = 0.f;
    const int64_t col = me.group * P;
    auto load = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            const int64_t at = row * p.Dm + col + me.at(k);
            s[k] = load_vec<T, kVec, kLoose>(static_cast<const T *>(p.s) + at, n[k]);
            g[k] = load_vec<T, kVec, kLoose>(static_cast<const T *>(p.dy) + at, n[k]);
            if (p.dsum) r[k] = load_vec<T, kVec, kLoose>(static_cast<const T *>(p.dsum) + at, n[k]);
        }
        if (me.on) {
            mean = p.mean[row * ng + me.group];
            rstd = p.rstd[row * ng + me.group];
        }
    };
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        const int left = me.on ? P - me.at(k) : 0;
        n[k] = left < 0 ? 0 : left > kVec ? kVec : left;
    }
    if (kAhead) load(blockIdx.y);
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        load_params<kVec>(p.weight + col + me.at(k), p.weight != nullptr, n[k], 1.f, w[k]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) dw[k][e] = db[k][e] = 0.f;
    }
    const int waves = blockDim.x / kWave;
    int turn = 0, chain = 0;
    bool begun = false;  // the block's partial sums hold earlier chains
    // part: [row block][dweight, dbias][Dm]
    auto flush = [&] {
        float *dst = p.part + (int64_t)blockIdx.y * 2 * p.Dm;
        const int Dm = (int)p.Dm;
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            int at = (int)col + me.at(k);
            asm volatile("" : "+v"(at));  // computed here, not kept across the rows
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (has(k, e)) {
                    float *to_w = dst + (at + e), *to_b = to_w + Dm;
                    *to_w = begun ? *to_w + dw[k][e] : dw[k][e];
                    *to_b = begun ? *to_b + db[k][e] : db[k][e];
                    dw[k][e] = db[k][e] = 0.f;
                }
        }
        begun = true;
        chain = 0;
    };
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const int64_t base = row * p.Dm + col;
        if (!kAhead) load(row);
        float z[kNv][kVec], q[kNv][kVec], a = 0.f, b = 0.f;
        Stored<T, kVec> d[kNv];
        const float scale = rstd;
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            d[k] = r[k];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float dy = to_f32(g[k].v[e]);
                z[k][e] = has(k, e) ? (to_f32(s[k].v[e]) - mean) * rstd : 0.f;
                q[k][e] = dy * w[k][e];
                a += q[k][e];
                b = __builtin_fmaf(q[k][e], z[k][e], b);
                dw[k][e] = __builtin_fmaf(dy, z[k][e], dw[k][e]);
                db[k][e] += dy;
            }
        }
        if (kAhead && row + gridDim.y < p.rows) load(row + gridDim.y);
        a = lanes_sum<kLanes>(a);
        b = lanes_sum<kLanes>(b);
        if constexpr (kTeam == 0) {
            if (waves > 1) {
                if (lane == 0) {
                    red[turn][wave][0] = a;
                    red[turn][wave][1] = b;
                }
                __syncthreads();
                a = uniform_f(lanes_sum<kNormMaxWaves>(lane < waves ? red[turn][lane % kNormMaxWaves][0] : 0.f));
                b = uniform_f(lanes_sum<kNormMaxWaves>(lane < waves ? red[turn][lane % kNormMaxWaves][1] : 0.f));
                turn ^= 1;
            }
        }
        a *= inv;
        b *= inv;
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            Stored<T, kVec> out;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float v = scale * (q[k][e] - a - z[k][e] * b);
                out.v[e] = from_acc<T>(p.dsum ? v + to_f32(d[k].v[e]) : v);
            }
            store_vec<T, kVec, kLoose>(static_cast<T *>(p.dx) + base + me.at(k), n[k], out);
        }
        if (++chain == kNormSumRows && p.part != nullptr && row + gridDim.y < p.rows) flush();
    }
    if (p.part != nullptr) flush();
}

// Groups too long for a block's registers (2048 vectors): a block takes one group
// after another and reads its values again for each step (from the caches, as far as
// they hold), one by one.  8192 x 12288 fp32 403 us forward and 465 backward, 2.4
// and 1.9 times its bytes' time; 8192 x 20480 bf16 596 and 634, 4.3 and 3.1 times.
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = lanes_sum<64>(v);
    __syncthreads();  // (red may still be read from the sum before)
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int z = 0; z < 16; ++z) t += red[z];
    return t;
}

template <typename T>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(NormParams p) {
    __shared__ float red[16];
    const int64_t ng = p.Dm / p.group;
    const int P = (int)p.group, tid = threadIdx.x;
    for (int64_t id = blockIdx.x; id < p.rows * ng; id += gridDim.x) {
        const int64_t col = id % ng * P, base = id / ng * p.Dm + col;
        const T *x = static_cast<const T *>(p.x) + base;
        const T *res = p.residual ? static_cast<const T *>(p.residual) + base : nullptr;
        T *sum = p.sum ? static_cast<T *>(p.sum) + base : nullptr;
        T *y = static_cast<T *>(p.y) + base;
        // (the sum may replace the residual: each value is read for the last
        // time by the thread that then writes it)
        auto value = [&](int c) { return res ? to_f32(from_acc<T>(to_f32(x[c]) + to_f32(res[c]))) : to_f32(x[c]); };
        float a = 0.f;
        for (int c = tid; c < P; c += 1024) a += value(c);
        const float mean = block_sum(a, red) / (float)P;
        float b = 0.f;
        for (int c = tid; c < P; c += 1024) {
            const float v = value(c) - mean;
            b = __builtin_fmaf(v, v, b);
        }
        const float rstd = 1.0f / sqrtf(block_sum(b, red) / (float)P + p.eps);
        for (int c = tid; c < P; c += 1024) {
            const float v = value(c);
            const float w = p.weight ? p.weight[col + c] : 1.f;
            const float o = p.bias ? p.bias[col + c] : 0.f;
            y[c] = from_acc<T>(__builtin_fmaf((v - mean) * rstd, w, o));
            if (sum) sum[c] = from_acc<T>(v);
        }
        if (tid == 0) {
            if (p.mean) p.mean[id] = mean;
            if (p.rstd) p.rstd[id] = rstd;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(NormBwdParams p) {
    __shared__ float red[16];
    const int64_t ng = p.Dm / p.group;
    const int P = (int)p.group, tid = threadIdx.x;
    for (int64_t id = blockIdx.x; id < p.rows * ng; id += gridDim.x) {
        const int64_t col = id % ng * P, base = id / ng * p.Dm + col;
        const T *s = static_cast<const T *>(p.s) + base, *dy = static_cast<const T *>(p.dy) + base;
        const T *dsum = p.dsum ? static_cast<const T *>(p.dsum) + base : nullptr;
        T *dx = static_cast<T *>(p.dx) + base;
        const float *w = p.weight ? p.weight + col : nullptr;
        const float mean = p.mean[id], rstd = p.rstd[id];
        float a = 0.f, b = 0.f;
        for (int c = tid; c < P; c += 1024) {
            const float q = to_f32(dy[c]) * (w ? w[c] : 1.f);
            a += q;
            b = __builtin_fmaf(q, (to_f32(s[c]) - mean) * rstd, b);
        }
        a = block_sum(a, red) / (float)P;
        b = block_sum(b, red) / (float)P;
        for (int c = tid; c < P; c += 1024) {
            const float q = to_f32(dy[c]) * (w ? w[c] : 1.f);
            const float z = (to_f32(s[c]) - mean) * rstd;
            dx[c] = from_acc<T>(rstd * (q - a - z * b) + (dsum ? to_f32(dsum[c]) : 0.f));
        }
    }
}

// dweight and dbias of a block of rows for those groups: one thread per
// channel, part[row block][dweight, dbias][Dm].
template <typename T>
__global__ __launch_bounds__(256) void norm_bwd_long_sum_kernel(NormBwdParams p) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= p.Dm) return;
    const int64_t ng = p.Dm / p.group, gr = c / p.group;
    const T *s = static_cast<const T *>(p.s), *dy = static_cast<const T *>(p.dy);
    float dw = 0.f, db = 0.f, dw_all = 0.f, db_all = 0.f;
    int chain = 0;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float v = to_f32(dy[row * p.Dm + c]);
        dw = __builtin_fmaf(v, (to_f32(s[row * p.Dm + c]) - p.mean[row * ng + gr]) * p.rstd[row * ng + gr], dw);
        db += v;
        if (++chain == kNormSumRows) {
            dw_all += dw;
            db_all += db;
            dw = db = 0.f;
            chain = 0;
        }
    }
    p.part[(int64_t)blockIdx.y * 2 * p.Dm + c] = dw_all + dw;
    p.part[(int64_t)blockIdx.y * 2 * p.Dm + p.Dm + c] = db_all + db;
}

// dweight and dbias from `blocks` rows of partial sums: a block of 16 waves
// adds 64 channels, each wave every 16th row, then across the waves.
__global__ __launch_bounds__(1024) static void norm_sum_kernel(const float *__restrict__ part, int blocks, int64_t Dm,
                                                               float *__restrict__ dweight, float *__restrict__ dbias) {
    __shared__ float red[16][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWave + lane;
    float *out = blockIdx.y == 0 ? dweight : dbias;
    if (out == nullptr) return;
    const float *src = part + (blockIdx.y == 0 ? 0 : Dm) + c;
    float s = 0.f;
    if (c < Dm) {
        int r = wave;
        for (; r + 7 * 16 < blocks; r += 8 * 16) {
            float t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = src[(int64_t)(r + k * 16) * 2 * Dm];
#pragma unroll
            for (int k = 0; k < 8; ++k) s += t[k];
        }
        for (; r < blocks; r += 16) s += src[(int64_t)r * 2 * Dm];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < Dm) {
        float t = 0.f;
#pragma unroll
        for (int z = 0; z < 16; ++z) t += red[z][lane];
        out[c] = t;
    }
}

// ---------------------------------------------------------------------------
// Launching.

// Row blocks of a grid: as many blocks as the chip holds at once, so that they
// all walk the same number of rows side by side (one block more per CU would
// run alone after the others: 1.16 against 1.04 ms at 65536 x 5120), and no more
// partial sums of the parameters' gradients than that.  held: waves a CU holds of
// the kernel.
inline unsigned norm_row_blocks(int64_t rows, int64_t col_blocks, int waves, int held, int cus) {
    const int64_t all = (int64_t)cus * (held / waves > 1 ? held / waves : 1);
    const int64_t most = all / col_blocks > 1 ? all / col_blocks : 1;
    return (unsigned)(rows < most ? rows : most);
}
// Those waves by the registers that the compiler gives the kernels, of lanes with
// one vector (with two, half as many).  They follow a change of the kernels or of
// the compiler only by hand; tests/test_kernel_resources_cpu.py compares.  A kernel
// that held fewer would take longer, with the same results.
constexpr int kNormFwdHeld = 32;
template <typename T>
constexpr int kNormBwdHeld = sizeof(T) == 4 ? 32 : 20;

// The backward's: also at least eight rows to a block where that leaves one for
// every CU, since each block writes a row of partial sums.
inline unsigned norm_bwd_row_blocks(int64_t rows, int64_t col_blocks, int waves, int held, int cus) {
    const int64_t few = (rows + 7) / 8 > cus ? (rows + 7) / 8 : cus;
    const int64_t n = norm_row_blocks(rows, col_blocks, waves, held, cus);
    return (unsigned)(n < few ? n : few);
}

template <int N>
struct Int {
    static constexpr int value = N;
};

// Calls f(team, vectors per lane, threads of a block) with the shape for groups
// of P channels.  Returns false when a group does not fit a block's registers.
template <typename T, typename F>
bool norm_shape(int64_t P, F f) {
    constexpr int W = 16 / (int)sizeof(T);
    auto lanes = [](int64_t n) { return (int)((n + kWave - 1) / kWave * kWave); };
    const int64_t n = (P + W - 1) / W;
    if (n <= 8) f(Int<8>(), Int<1>(), 256);
    else if (n <= 16) f(Int<16>(), Int<1>(), 256);
    else if (n <= 32) f(Int<32>(), Int<1>(), 256);
    else if (n <= 64) f(Int<64>(), Int<1>(), 256);
    else if (n <= 1024) f(Int<0>(), Int<1>(), lanes(n));
    else if (n <= 2048) f(Int<0>(), Int<2>(), lanes((n + 1) / 2));
    else return false;
    return true;
}

// Blocks across a row of ng groups.
inline int64_t norm_col_blocks(int64_t ng, int team) {
    const int per = team ? 256 / team : 1;
    return (ng + per - 1) / per;
}

inline bool norm_aligned(const void *const *ptrs, int n) {
    uintptr_t bits = 0;
    for (int k = 0; k < n; ++k) bits |= (uintptr_t)ptrs[k];
    return bits % 16 == 0;
}

inline unsigned norm_long_blocks(int64_t groups) { return (unsigned)(groups < 65536 ? groups : 65536); }

// Whether every vector is whole and aligned.
template <typename T>
bool norm_tight(int64_t group, const void *const *ptrs, int n) {
    return group % (16 / (int)sizeof(T)) == 0 && norm_aligned(ptrs, n);
}

template <typename T>
hipError_t norm_fwd_t(const NormParams &p, hipStream_t s) {
    const void *ptrs[] = {p.x, p.residual, p.sum, p.y};
    const bool tight = norm_tight<T>(p.group, ptrs, 4);
    const int64_t ng = p.Dm / p.group;
    const bool held = norm_shape<T>(p.group, [&](auto team, auto nv, int block) {
        constexpr int kTeam = decltype(team)::value, kNv = decltype(nv)::value, kVec = 16 / (int)sizeof(T);
        const int64_t cols = norm_col_blocks(ng, kTeam);
        const dim3 grid((unsigned)cols, norm_row_blocks(p.rows, cols, block / kWave, kNormFwdHeld / kNv, p.cus));
        if (tight)
            hipLaunchKernelGGL((norm_fwd_kernel<T, kVec, kTeam, kNv, false>), grid, dim3(block), 0, s, p);
        else
            hipLaunchKernelGGL((norm_fwd_kernel<T, kVec, kTeam, kNv, true>), grid, dim3(block), 0, s, p);
    });
    if (!held)
        hipLaunchKernelGGL(norm_fwd_long_kernel<T>, dim3(norm_long_blocks(p.rows * ng)), dim3(1024), 0, s, p);
    return hipGetLastError();
}

// Row blocks of the backward: the rows of its partial sums.
template <typename T>
unsigned norm_bwd_blocks(const NormBwdParams &p) {
    const int64_t ng = p.Dm / p.group;
    unsigned n = norm_bwd_row_blocks(p.rows, (p.Dm + 255) / 256, 4, 32, p.cus);
    norm_shape<T>(p.group, [&](auto team, auto nv, int block) {
        n = norm_bwd_row_blocks(p.rows, norm_col_blocks(ng, decltype(team)::value), block / kWave,
                                kNormBwdHeld<T> / decltype(nv)::value, p.cus);
    });
    return n;
}

template <typename T>
hipError_t norm_bwd_t(NormPass pass, NormBwdParams &p, size_t *bytes, hipStream_t s) {
    const void *ptrs[] = {p.s, p.dy, p.dsum, p.dx};
    const bool tight = norm_tight<T>(p.group, ptrs, 4);
    const unsigned blocks = norm_bwd_blocks<T>(p);
    const bool params = p.dweight != nullptr || p.dbias != nullptr;
    if (pass == NormPass::kPlan) {
        *bytes = params ? (size_t)blocks * 2 * (size_t)p.Dm * 4 : 0;
        return hipSuccess;
    }
    if (pass == NormPass::kReduce) {
        hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((p.Dm + kWave - 1) / kWave), 2), dim3(1024), 0, s, p.part,
                           (int)blocks, p.Dm, p.dweight, p.dbias);
        return hipGetLastError();
    }
    const int64_t ng = p.Dm / p.group;
    const bool held = norm_shape<T>(p.group, [&](auto team, auto nv, int block) {
        constexpr int kTeam = decltype(team)::value, kNv = decltype(nv)::value, kVec = 16 / (int)sizeof(T);
        const dim3 grid((unsigned)norm_col_blocks(ng, kTeam), blocks);
        if (tight)
            hipLaunchKernelGGL((norm_bwd_kernel<T, kVec, kTeam, kNv, false>), grid, dim3(block), 0, s, p);
        else
            hipLaunchKernelGGL((norm_bwd_kernel<T, kVec, kTeam, kNv, true>), grid, dim3(block), 0, s, p);
    });
    if (!held) {
        hipLaunchKernelGGL(norm_bwd_long_kernel<T>, dim3(norm_long_blocks(p.rows * ng)), dim3(1024), 0, s, p);
        if (params)
            hipLaunchKernelGGL(norm_bwd_long_sum_kernel<T>, dim3((unsigned)((p.Dm + 255) / 256), blocks), dim3(256), 0,
                               s, p);
    }
    return hipGetLastError();
}

}  // namespace ssm
