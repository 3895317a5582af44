// Linear attention with one decay per head (gfx950): chunks of steps on the
// matrix cores, joined by the heads' states.
//
// A head with decay L = exp(a) has the state H (nv x nk) and
//   H_t = L H_{t-1} + v_t k_t^T,   y_t = H_t q_t.
// A chunk of C steps that starts from H is, with steps counted from 0,
//   y_t = L^{t+1} H q_t + sum_{s<=t} L^{t-s} (k_s . q_t) v_s
//   H'  = L^C H + sum_s L^{C-1-s} v_s k_s^T
// Every exponent is >= 0, so nothing grows for a <= 0.
//
// The gradients are the same operation with other arguments.  With the
// adjoint G_t = L G_{t+1} + dy_t q_t^T (dL/dH_t):
//   dq_t = H_t^T dy_t                     q, k, v <- dy, v, k; state H^T
//   dv_t = G_t k_t,  dh_init = L G_0      backwards in time, q, k, v <- k, q, dy; state G
//   dk_t = G_t^T v_t                      backwards in time, q, k, v <- v, dy, q; state G^T
// Backwards, the chunk's rows are loaded in reverse order.  dh_final enters G
// undecayed: there the state that enters counts as L^t and the sum of the
// state that leaves as L^{C-s}.
//
// Layout of work: a block of one wave per 32 columns of v takes one head of a
// part of a sequence, chunk after chunk; each wave keeps its columns of the
// state in accumulators (nk x 32).  The four products -- S = k q^T, S v, H q
// and v k^T -- are 32x32 tiles: bf16 storage takes v_mfma_f32_32x32x16_bf16,
// with an fp32 operand (the weighted S, the state, the weighted v) as the sum of
// bf16 terms; fp32 storage takes v_mfma_f32_32x32x2_f32.  Matrix rows are dealt
// to lanes with bits 2 and 3 exchanged (lin_row), so that the 8 accumulators of a lane
// are 8 consecutive rows: an accumulator tile becomes an operand in place, row
// operands are 16-byte LDS reads, and y leaves as 16-byte stores.
#pragma once

#include <type_traits>

#include "attn_launch.h"
#include "ssm_device.h"

namespace ssm {

typedef __bf16 lin_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 lin_bf16x2 __attribute__((ext_vector_type(2)));
typedef float lin_f32x2 __attribute__((ext_vector_type(2)));
typedef float lin_f32x4 __attribute__((ext_vector_type(4)));
typedef float lin_f32x16 __attribute__((ext_vector_type(16)));
typedef short lin_i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) lin_i16x4 lin_lds_i16x4;

// Chunk length: two 32-step tiles for bf16 storage.  One where the registers
// that stage the next chunk would not fit (few waves to a wide q and k), and for
// fp32 storage, which spends nothing on splitting the state and gains by the
// smaller S.
template <typename T, int NK, int NV>
constexpr int lin_steps() { return sizeof(T) == 4 || NK > NV ? 32 : 64; }
// Terms of an fp32 operand of a product: y from two bf16 terms (2^-18 of an
// operand), the states from three (2^-26), as they are kept in fp32.
template <typename T> constexpr int lin_terms() { return sizeof(T) == 4 ? 1 : 2; }
template <typename T> constexpr int lin_state_terms() { return sizeof(T) == 4 ? 1 : 3; }

// An operand of a product over 16 values of k: lane l holds row (or column)
// l % 32, its slot e the value k0 + 8 (l / 32) + e.
template <typename T>
struct LinFrag;
template <>
struct LinFrag<bf16> {
    lin_bf16x8 v;
};
template <>
struct LinFrag<float> {
    float v[8];
};
__device__ __forceinline__ void lin_mma(lin_f32x16 &acc, const LinFrag<bf16> &a, const LinFrag<bf16> &b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void lin_mma(lin_f32x16 &acc, const LinFrag<float> &a, const LinFrag<float> &b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[e], b.v[e], acc, 0, 0, 0);
}

// v as a sum of kTerms stored values, each the rounding of what is left.
template <int kTerms>
__device__ __forceinline__ void lin_split(float (&v)[8], LinFrag<bf16> (&f)[kTerms]) {
#pragma unroll
    for (int n = 0; n < kTerms; ++n) {
        u32x4 h;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const lin_f32x2 ab = {v[2 * k], v[2 * k + 1]};
            h[k] = __builtin_bit_cast(unsigned, __builtin_convertvector(ab, lin_bf16x2));
            if (n + 1 < kTerms) {
                v[2 * k] -= __builtin_bit_cast(float, h[k] << 16);
                v[2 * k + 1] -= __builtin_bit_cast(float, h[k] & 0xffff0000u);
            }
        }
        f[n].v = __builtin_bit_cast(lin_bf16x8, h);
    }
}
template <int kTerms>
__device__ __forceinline__ void lin_split(float (&v)[8], LinFrag<float> (&f)[kTerms]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[0].v[e] = v[e];
}
__device__ __forceinline__ float lin_elem(const LinFrag<bf16> &f, int e) { return static_cast<float>(f.v[e]); }
__device__ __forceinline__ float lin_elem(const LinFrag<float> &f, int e) { return f.v[e]; }

// The matrix row that lane l % 32 (and accumulator row l % 32) stands for:
// bits 2 and 3 exchanged.  Register 8 j + e of lane group g is row 16 j + 8 g + e.
__device__ __forceinline__ int lin_row(int l) { return (l & 0x13) | ((l & 4) << 1) | ((l & 8) >> 1); }

// Rows in LDS: granules of 16 bytes, kG to a row, without padding.  The
// granules of a row are exchanged by a pattern of the row, so that 8 rows read
// at one granule, and 4 rows read at 4 granules (the transposing reads), fall on
// different banks.
template <int kG>
__device__ __forceinline__ int lin_at(int row, int c) {
    constexpr int kLines = 16 / (kG < 16 ? kG : 16);  // rows that share 256 bytes
    const int f = (((row / kLines) & (kG / 4 - 1)) << 2) | ((row >> 2) & 3);
    return row * kG + (c ^ (f & (kG - 1)));
}

// The operand of row `row`, values k0 + 8 g + (0..7).
template <int N>
__device__ __forceinline__ void lin_row_frag(LinFrag<bf16> &f, const u32x4 *t, int row, int k0, int g) {
    f.v = __builtin_bit_cast(lin_bf16x8, t[lin_at<N / 8>(row, k0 / 8 + g)]);
}
template <int N>
__device__ __forceinline__ void lin_row_frag(LinFrag<float> &f, const u32x4 *t, int row, int k0, int g) {
    const u32x4 a = t[lin_at<N / 4>(row, k0 / 4 + 2 * g)], b = t[lin_at<N / 4>(row, k0 / 4 + 2 * g + 1)];
    __builtin_memcpy(&f.v[0], &a, 16);
    __builtin_memcpy(&f.v[4], &b, 16);
}
// The operand of column c0 + lin_row(lane % 32), rows s0 + 8 g + (0..7).  bf16:
// two transposing LDS loads, in which, of 16 lanes, lane m addresses four
// columns of row m / 4 and lane i receives column i of the four rows.
template <int N>
__device__ __forceinline__ void lin_col_frag(LinFrag<bf16> &f, const u32x4 *t, int s0, int c0, int lane) {
    const int row = s0 + 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int c = c0 / 8 + 2 * ((lane >> 4) & 1) + (lane & 1), half = (lane >> 1) & 1;
    auto at = [&](int r) {
        return (lin_lds_i16x4 *)(reinterpret_cast<const char *>(t + lin_at<N / 8>(r, c)) + 8 * half);
    };
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(row)));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(row + 4)));
    const u32x4 u = {a.x, a.y, b.x, b.y};
    f.v = __builtin_bit_cast(lin_bf16x8, u);
}
template <int N>
__device__ __forceinline__ void lin_col_frag(LinFrag<float> &f, const u32x4 *t, int s0, int c0, int lane) {
    const int col = c0 + lin_row(lane & 31);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f.v[e] = reinterpret_cast<const float *>(t + lin_at<N / 4>(s0 + 8 * (lane >> 5) + e, col / 4))[col % 4];
}

// A barrier for handing LDS between waves that does not wait for loads from
// memory in flight (__syncthreads does).
__device__ __forceinline__ void lin_barrier() {
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// A chunk's rows of one tensor on their way through registers to LDS: granule
// i * kThreads + tid of the tile.
template <typename T, int N, int kC, int kThreads>
struct LinTile {
    static constexpr int kG = N * (int)sizeof(T) / 16, kCount = kC * kG / kThreads;
    static_assert(kC * kG % kThreads == 0, "whole granules per thread");
    u32x4 r[kCount];
    // `base`: the head's values of the lowest step of the chunk, steps `stride` bytes apart, `width` of N values
    __device__ __forceinline__ void load(const char *base, int32_t stride, int width, int rows, bool reverse) {
        const __amdgpu_buffer_rsrc_t d =
            make_rsrc(base, (int32_t)((rows - 1) * stride + width * (int)sizeof(T)));
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int at = i * kThreads + (int)threadIdx.x, row = at / kG, c = at % kG;
            const int step = reverse ? rows - 1 - row : row;
            const bool in = row < rows && c * 16 < width * (int)sizeof(T);
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(d, in ? step * stride + c * 16 : 0x7fffffff, 0, 0);
        }
    }
    __device__ __forceinline__ void store(u32x4 *t) const {
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int at = i * kThreads + (int)threadIdx.x;
            t[lin_at<kG>(at / kG, at % kG)] = r[i];
        }
    }
};

// Where a block works.
struct LinPlace {
    int64_t begin, end;  // steps of its sequence
    int64_t from, count; // its own, counted in the direction of the pass
    int64_t part;        // its entry of the parts' states
    int row;             // sequence (or batch row)
    bool first, last;
};
__device__ __forceinline__ bool lin_place(const LinParams &p, int64_t part, LinPlace &me) {
    int64_t index;
    if (p.table) {
        const LinSeg s = p.table[part];
        if (s.index < 0) return false;
        me.begin = s.begin, me.end = s.end, me.row = s.seq, index = s.index;
    } else {
        const int64_t per = p.segs / p.Bsz;
        me.row = (int)(part / per);
        index = part - me.row * per;
        me.begin = me.row * p.L, me.end = me.begin + p.L;
    }
    me.part = part;
    me.from = index * p.seg_len;
    const int64_t left = me.end - me.begin - me.from;
    me.count = left < p.seg_len ? left : p.seg_len;
    me.first = index == 0, me.last = left <= p.seg_len;
    return left > 0;
}

// A wave's columns of a state: register 8 j + e of tile nt of lane (col, g) is
// row 32 nt + 16 j + 8 g + e.
template <int NK, typename F>
__device__ __forceinline__ void lin_each_run(int g, F f) {
#pragma unroll
    for (int nt = 0; nt < NK / 32; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) f(nt, 8 * j, 32 * nt + 16 * j + 8 * g);
}
template <int NK>
__device__ __forceinline__ void lin_state_load(lin_f32x16 (&h)[NK / 32], const float *src, int sn, int nk, int g,
                                               bool col_ok) {
    lin_each_run<NK>(g, [&](int nt, int r, int n) {
        if (sn == 1) {
            lin_f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
            if (col_ok && n < nk) {  // nk is a multiple of 8
                a = *reinterpret_cast<const lin_f32x4 *>(src + n);
                b = *reinterpret_cast<const lin_f32x4 *>(src + n + 4);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) h[nt][r + e] = a[e], h[nt][r + 4 + e] = b[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[nt][r + e] = col_ok && n < nk ? src[(int64_t)(n + e) * sn] : 0.f;
        }
    });
}
template <int NK>
__device__ __forceinline__ void lin_state_store(const lin_f32x16 (&h)[NK / 32], float *dst, int sn, int nk, int g,
                                                bool col_ok) {
    lin_each_run<NK>(g, [&](int nt, int r, int n) {
        if (!col_ok || n >= nk) return;
        if (sn == 1) {
            lin_f32x4 a, b;
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = h[nt][r + e], b[e] = h[nt][r + 4 + e];
            *reinterpret_cast<lin_f32x4 *>(dst + n) = a;
            *reinterpret_cast<lin_f32x4 *>(dst + n + 4) = b;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[(int64_t)(n + e) * sn] = h[nt][r + e];
        }
    });
}

// The log decay in base-2 units.  Below -1e4 every power but the 0th is 0
// (and 0 times it stays 0: a = -inf is a state without memory).
__device__ __forceinline__ float lin_log2_decay(float a) {
    const float a2 = a * kLog2e;
    return a2 < -1e4f ? -1e4f : a2;
}

// kOut: y of every step, and the last part's state to h_final.  Otherwise the
// state that a part adds (from zero) to the next part's entry of `states`.
template <typename T, int NK, int NV, bool kOut>
__global__ __launch_bounds__(2 * NV, 2) void lin_chunk_kernel(LinParams p) {
    constexpr int kC = lin_steps<T, NK, NV>(), kTT = kC / 32, kThreads = 2 * NV, kWaves = NV / 32;
    constexpr int kGK = NK * (int)sizeof(T) / 16, kGV = NV * (int)sizeof(T) / 16;
    constexpr int kTerms = lin_terms<T>(), kStateTerms = lin_state_terms<T>();
    constexpr int kTiles = kTT == 2 ? 3 : 1;                // causal tiles of S
    constexpr int kFragWords = (int)sizeof(LinFrag<T>) / 16;  // 16-byte words of a fragment
    __shared__ __attribute__((aligned(16))) u32x4 lq[kOut ? kC * kGK : 1];
    __shared__ __attribute__((aligned(16))) u32x4 lk[kC * kGK];
    __shared__ __attribute__((aligned(16))) u32x4 lv[kC * kGV];
    __shared__ __attribute__((aligned(16))) u32x4 ls[kOut ? kTiles * 2 * kTerms * kFragWords * kWave : 1];
    __shared__ __attribute__((aligned(16))) float lw[kC];

    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const int g = lane >> 5, li = lane & 31;
    const int block = xcd_remap(blockIdx.x, gridDim.x);
    const int h = block % p.H;
    LinPlace me;
    if (!lin_place(p, block / p.H, me)) return;
    if (!kOut && me.last) return;

    const float a2 = lin_log2_decay(p.log_decay[h]);
    const int off = p.reverse ? 0 : 1;  // decays of an entering state at its first step
    const int col = 32 * wave + lin_row(li);
    const bool col_ok = col < p.nv;
    const int64_t state = (int64_t)p.nk * p.nv;

    lin_f32x16 hs[NK / 32];
    const float *src = nullptr;
    int sn = 1;
    if constexpr (kOut) {
        if (!me.first || (p.states && p.copy_first))
            src = p.states + (me.part * p.H + h) * state + (int64_t)col * p.nk;
        else if (p.h_init)
            src = p.h_init + ((int64_t)me.row * p.H + h) * state + (int64_t)col * p.sc, sn = p.sn;
    }
    if (src) {
        lin_state_load<NK>(hs, src, sn, p.nk, g, col_ok);
    } else {
#pragma unroll
        for (int nt = 0; nt < NK / 32; ++nt)
#pragma unroll
            for (int r = 0; r < 16; ++r) hs[nt][r] = 0.f;
    }

    // ---- the tensors' rows
    const int32_t es = sizeof(T);
    const int32_t q_step = (p.H / p.gq) * p.nk * es, k_step = (p.H / p.gk) * p.nk * es, v_step = (p.H / p.gv) * p.nv * es;
    const int chunks = (int)((me.count + kC - 1) / kC);
    auto rows_of = [&](int c) { return (int)(me.count - (int64_t)c * kC < kC ? me.count - (int64_t)c * kC : kC); };
    auto lowest = [&](int c) {  // step in memory of the chunk's lowest row
        const int64_t at = me.from + (int64_t)c * kC;
        return p.reverse ? me.end - at - rows_of(c) : me.begin + at;
    };
    LinTile<T, NK, kC, kThreads> tq, tk;
    LinTile<T, NV, kC, kThreads> tv;
    auto fetch = [&](int c) {
        const int64_t at = lowest(c);
        const int rows = rows_of(c);
        if constexpr (kOut)
            tq.load(static_cast<const char *>(p.q) + at * q_step + (int64_t)(h / p.gq) * p.nk * es, q_step, p.nk, rows,
                    p.reverse);
        tk.load(static_cast<const char *>(p.k) + at * k_step + (int64_t)(h / p.gk) * p.nk * es, k_step, p.nk, rows,
                p.reverse);
        tv.load(static_cast<const char *>(p.v) + at * v_step + (int64_t)(h / p.gv) * p.nv * es, v_step, p.nv, rows,
                p.reverse);
    };
    // the staged rows to LDS, and the weights of the chunk's rows in the state
    // (rows past its end are zeros)
    auto place = [&](int c) {
        if constexpr (kOut) tq.store(lq);
        tk.store(lk);
        tv.store(lv);
        const int back = rows_of(c) - off - (int)threadIdx.x;
        if (threadIdx.x < kC && (c == 0 || rows_of(c) != kC))
            lw[threadIdx.x] = back >= 0 ? fast_exp2((float)back * a2) * p.k_scale : 0.f;
    };

    // ---- weights L^{t-s} of this wave's tiles of S, 0 above the diagonal: waves
    // 0 and 2 have diagonal tiles, wave 1 the one below
    float weight[kOut ? 16 : 1];
    float fade[kTT];  // L^{t + off} of this lane's steps
    const bool below = kTT == 2 && wave == 1;
    if constexpr (kOut) {
        const float sc = p.y_scale * p.k_scale;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int back = li - (16 * (r / 8) + 8 * g + r % 8) + (below ? 32 : 0);
            weight[r] = back >= 0 ? fast_exp2((float)back * a2) * sc : 0.f;
        }
#pragma unroll
        for (int tt = 0; tt < kTT; ++tt) fade[tt] = fast_exp2((float)(32 * tt + li + off) * a2) * p.y_scale;
    }

    fetch(0);
    place(0);
    lin_barrier();
    for (int c = 0; c < chunks; ++c) {
        const bool more = c + 1 < chunks;
        const int rows = rows_of(c);
        if (more) fetch(c + 1);
        LinFrag<T> vf[kC / 16];
#pragma unroll
        for (int j = 0; j < kC / 16; ++j) lin_col_frag<NV>(vf[j], lv, 16 * j, 32 * wave, lane);
        lin_f32x16 y[kOut ? kTT : 1];
        if constexpr (kOut) {
            // ---- S^T = k q^T of the causal tiles (rows s, columns t), weighted, to LDS as operands
#pragma unroll
            for (int tile = 0; tile < kTiles; ++tile) {
                if (kWaves >= 4 ? wave != tile : (wave == 1) != (tile == 1)) continue;
                const int st = tile / 2, tt = (tile + 1) / 2;
                lin_f32x16 s;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = 0.f;
#pragma unroll
                for (int k0 = 0; k0 < NK; k0 += 16) {
                    LinFrag<T> kf, qf;
                    lin_row_frag<NK>(kf, lk, 32 * st + lin_row(li), k0, g);
                    lin_row_frag<NK>(qf, lq, 32 * tt + li, k0, g);
                    lin_mma(s, kf, qf);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float w[8];
                    LinFrag<T> f[kTerms];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const bool in = st != tt || 16 * j + 8 * g + e <= li;
                        w[e] = in ? s[8 * j + e] * weight[8 * j + e] : 0.f;
                    }
                    lin_split<kTerms>(w, f);
#pragma unroll
                    for (int n = 0; n < kTerms; ++n) {
                        u32x4 u[kFragWords];
                        __builtin_memcpy(u, &f[n], sizeof u);
#pragma unroll
                        for (int k = 0; k < kFragWords; ++k)
                            ls[(((tile * 2 + j) * kTerms + n) * kFragWords + k) * kWave + lane] = u[k];
                    }
                }
            }
            // ---- y^T = H q^T (rows of v's columns, columns t)
#pragma unroll
            for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
                for (int r = 0; r < 16; ++r) y[tt][r] = 0.f;
#pragma unroll
            for (int k0 = 0; k0 < NK; k0 += 16) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = hs[k0 / 32][8 * (k0 / 16 % 2) + e];
                LinFrag<T> hf[kTerms], qf[kTT];
                lin_split<kTerms>(v, hf);
#pragma unroll
                for (int tt = 0; tt < kTT; ++tt) lin_row_frag<NK>(qf[tt], lq, 32 * tt + li, k0, g);
#pragma unroll
                for (int n = 0; n < kTerms; ++n)
#pragma unroll
                    for (int tt = 0; tt < kTT; ++tt) lin_mma(y[tt], hf[n], qf[tt]);
            }
#pragma unroll
            for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
                for (int r = 0; r < 16; ++r) y[tt][r] *= fade[tt];
        }
        // ---- H = L^rows H + sum of weighted v k^T.  A decay near 1 is applied by
        // its difference from 1: rounded to fp32 itself, it would be off by the same
        // 2^-25 at every chunk of a long memory.
        {
            const float z = (float)rows * a2;
            if (z > -1.f) {
                const float m = expm1f(z * 0.6931471805599453f);
#pragma unroll
                for (int nt = 0; nt < NK / 32; ++nt)
#pragma unroll
                    for (int r = 0; r < 16; ++r) hs[nt][r] = fma_(hs[nt][r], m, hs[nt][r]);
            } else {
                const float m = fast_exp2(z);
#pragma unroll
                for (int nt = 0; nt < NK / 32; ++nt)
#pragma unroll
                    for (int r = 0; r < 16; ++r) hs[nt][r] *= m;
            }
        }
#pragma unroll
        for (int j = 0; j < kC / 16; ++j) {
            float w[8];
            const lin_f32x4 a = *reinterpret_cast<const lin_f32x4 *>(lw + 16 * j + 8 * g);
            const lin_f32x4 b = *reinterpret_cast<const lin_f32x4 *>(lw + 16 * j + 8 * g + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = lin_elem(vf[j], e) * (e < 4 ? a[e % 4] : b[e % 4]);
            LinFrag<T> wf[kStateTerms];
            lin_split<kStateTerms>(w, wf);
#pragma unroll
            for (int nt = 0; nt < NK / 32; ++nt) {
                LinFrag<T> kf;
                lin_col_frag<NK>(kf, lk, 16 * j, 32 * nt, lane);
#pragma unroll
                for (int n = 0; n < kStateTerms; ++n) lin_mma(hs[nt], kf, wf[n]);
            }
        }
        lin_barrier();  // S is written; every wave is done with the chunk's rows
        if (more) place(c + 1);
        if constexpr (kOut) {
            // ---- y^T += v^T S^T
#pragma unroll
            for (int tile = 0; tile < kTiles; ++tile) {
                const int st = tile / 2, tt = (tile + 1) / 2;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int n = 0; n < kTerms; ++n) {
                        u32x4 u[kFragWords];
#pragma unroll
                        for (int k = 0; k < kFragWords; ++k)
                            u[k] = ls[(((tile * 2 + j) * kTerms + n) * kFragWords + k) * kWave + lane];
                        LinFrag<T> f;
                        __builtin_memcpy(&f, u, sizeof u);
                        lin_mma(y[tt], vf[2 * st + j], f);
                    }
            }
            // ---- y out: 8 consecutive values of a step per lane and half
            const int32_t ys = p.y_f32 ? 4 : es, y_step = p.H * p.nv * ys;
            const __amdgpu_buffer_rsrc_t d =
                make_rsrc(static_cast<char *>(p.y) + lowest(c) * y_step + (int64_t)h * p.nv * ys,
                          (rows - 1) * y_step + p.nv * ys);
#pragma unroll
            for (int tt = 0; tt < kTT; ++tt) {
                const int row = 32 * tt + li, step = p.reverse ? rows - 1 - row : row;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = 32 * wave + 16 * j + 8 * g;
                    const int32_t to = row < rows && at < p.nv ? step * y_step + at * ys : 0x7fffffff;
                    if (sizeof(T) == 4 || p.y_f32) {
                        u32x4 a, b;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            a[e] = __float_as_uint(y[tt][8 * j + e]);
                            b[e] = __float_as_uint(y[tt][8 * j + 4 + e]);
                        }
                        __builtin_amdgcn_raw_buffer_store_b128(a, d, to, 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b128(b, d, to, 16, 0);
                    } else {
                        u32x4 u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const lin_f32x2 v = {y[tt][8 * j + 2 * e], y[tt][8 * j + 2 * e + 1]};
                            u[e] = __builtin_bit_cast(unsigned, __builtin_convertvector(v, lin_bf16x2));
                        }
                        __builtin_amdgcn_raw_buffer_store_b128(u, d, to, 0, 0);
                    }
                }
            }
        }
        lin_barrier();  // the next chunk's rows are in, S is read
    }
    if constexpr (kOut) {
        if (me.last && p.h_final != nullptr)
            lin_state_store<NK>(hs, p.h_final + ((int64_t)me.row * p.H + h) * state + (int64_t)col * p.sc, p.sn, p.nk,
                                g, col_ok);
    } else {
        lin_state_store<NK>(hs, p.states + ((me.part + 1) * p.H + h) * state + (int64_t)col * p.nk, 1, p.nk, g, col_ok);
    }
}

template <typename T, int NK, int NV>
hipError_t lin_pass_n(LinPass pass, const LinParams &p, hipStream_t s) {
    const dim3 grid((unsigned)(p.segs * p.H));
    if (pass == LinPass::kAggregate)
        hipLaunchKernelGGL((lin_chunk_kernel<T, NK, NV, false>), grid, dim3(2 * NV), 0, s, p);
    else
        hipLaunchKernelGGL((lin_chunk_kernel<T, NK, NV, true>), grid, dim3(2 * NV), 0, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t lin_pass_t(LinPass pass, const LinParams &p, hipStream_t s) {
    if (p.nv <= 64) return p.nk <= 64 ? lin_pass_n<T, 64, 64>(pass, p, s) : lin_pass_n<T, 128, 64>(pass, p, s);
    return p.nk <= 64 ? lin_pass_n<T, 64, 128>(pass, p, s) : lin_pass_n<T, 128, 128>(pass, p, s);
}

// One decode step: h = L h + v k^T and y = scale h q.  A wave takes 8 rows of a
// state at a time (kRows of them, one behind the other), 8 lanes to a row; a
// lane holds four values of every 32.  Bound by the state's bytes.
constexpr int kLinStepRows = 2;
template <typename T, int kRuns>
__global__ __launch_bounds__(256) void lin_step_kernel(LinStepParams p) {
    const int lane = threadIdx.x % kWave, l8 = lane & 7;
    const int groups = (p.nv + 8 * kLinStepRows - 1) / (8 * kLinStepRows);
    const int64_t wave = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x / kWave);
    const int64_t bh = wave / groups;
    if (bh >= p.Bsz * p.H) return;
    const int64_t b = bh / p.H;
    const int h = (int)(bh - b * p.H), kv = h / p.group, kvs = p.H / p.group;
    const int row0 = (int)(wave - bh * groups) * 8 * kLinStepRows + lane / 8;
    const float *hs = p.h + bh * p.nv * p.nk;
    float *ho = p.h_out + bh * p.nv * p.nk;
    const T *q = static_cast<const T *>(p.q) + bh * p.nk;
    const T *k = static_cast<const T *>(p.k) + (b * kvs + kv) * p.nk;
    const T *v = static_cast<const T *>(p.v) + (b * kvs + kv) * p.nv;
    struct Four {
        T v[4];
    };
    lin_f32x4 st[kLinStepRows][kRuns];
#pragma unroll
    for (int u = 0; u < kLinStepRows; ++u)
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {
            const int n = 32 * j + 4 * l8, row = row0 + 8 * u;
            if (n < p.nk && row < p.nv)
                st[u][j] = __builtin_nontemporal_load(
                    reinterpret_cast<const lin_f32x4 *>(hs + (int64_t)row * p.nk + n));
        }
    float qv[kRuns][4], kk[kRuns][4], vv[kLinStepRows];
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
        const int n = 32 * j + 4 * l8;
        Four a{}, c{};
        if (n < p.nk) {
            __builtin_memcpy(&a, __builtin_assume_aligned(q + n, 4 * sizeof(T)), sizeof a);
            __builtin_memcpy(&c, __builtin_assume_aligned(k + n, 4 * sizeof(T)), sizeof c);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) qv[j][e] = to_f32(a.v[e]), kk[j][e] = to_f32(c.v[e]);
    }
#pragma unroll
    for (int u = 0; u < kLinStepRows; ++u) vv[u] = row0 + 8 * u < p.nv ? to_f32(v[row0 + 8 * u]) : 0.f;
    // a decay near 1 by its difference from 1: its own rounding would be a
    // wrong memory after many steps
    const float a = p.log_decay[h], m = a > -0.5f ? expm1f(a) : expf(a);
    const bool near1 = a > -0.5f;
#pragma unroll
    for (int u = 0; u < kLinStepRows; ++u) {
        const int row = row0 + 8 * u;
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {
            const int n = 32 * j + 4 * l8;
            if (n >= p.nk || row >= p.nv) continue;
            lin_f32x4 s = st[u][j];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[e] = fma_(vv[u], kk[j][e], near1 ? fma_(s[e], m, s[e]) : s[e] * m);
                y = fma_(s[e], qv[j][e], y);
            }
            __builtin_nontemporal_store(s, reinterpret_cast<lin_f32x4 *>(ho + (int64_t)row * p.nk + n));
        }
        y = lane_group_sum<8>(y);
        if (l8 == 0 && row < p.nv) static_cast<T *>(p.y)[bh * p.nv + row] = from_acc<T>(y * p.scale);
    }
}

template <typename T>
hipError_t lin_step_t(const LinStepParams &p, hipStream_t s) {
    const int groups = (p.nv + 8 * kLinStepRows - 1) / (8 * kLinStepRows);
    const dim3 grid((unsigned)((p.Bsz * p.H * groups + 3) / 4)), block(256);
    if (p.nk <= 32) hipLaunchKernelGGL((lin_step_kernel<T, 1>), grid, block, 0, s, p);
    else if (p.nk <= 64) hipLaunchKernelGGL((lin_step_kernel<T, 2>), grid, block, 0, s, p);
    else if (p.nk <= 96) hipLaunchKernelGGL((lin_step_kernel<T, 3>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((lin_step_kernel<T, 4>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace ssm
