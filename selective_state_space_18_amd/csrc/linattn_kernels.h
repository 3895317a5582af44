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
// Layout of work: a block takes one head of a part of a sequence, chunk after
// chunk; each wave keeps some columns (of v) of the state in accumulators.  An
// aggregate pass gives what every part adds to the state, from zero; an output pass
// runs the parts again from the states that enter them.  The products -- S = k q^T,
// S v, H q and v k^T -- are matrix-core tiles.  In bf16 storage an fp32 operand (the
// weighted S, the state, the weighted v) is the sum of bf16 terms, which multiply
// exactly.  Accumulators of a lane become an operand in place: products over them
// take their values in that order.
//   * bf16, output: lin_output_kernel, a wave per 32 columns, 32x32x16 tiles;
//   * bf16, aggregate, and fp32: lin_chunk_kernel, a wave per 16 columns, 16x16x32
//     (fp32 16x16x4) tiles.
// The wide tiles issue two thirds of the instructions (half the waves, so half of
// everything that is per wave) and read LDS half as often: output pass of 4 x 16384
// steps, 40 heads of 128, 745 -> 715 us when it came in (with two terms to an operand).  For
// the aggregate, whose state is most of its registers, they measured 271 us against 251.
//
// A chunk: its rows lie in LDS, written there from registers; the next chunk's loads set out
// when it begins.  S of the chunk is formed by some waves and handed to all
// through LDS; between, every wave adds H q and updates its state.  Two barriers a chunk.
//
// What bounds it (4 x 16384 steps, 40 heads of 128, bf16): output pass 707 to 808 us for 2.7 GB,
// 3.4 to 3.8 TB/s; matrix cores busy 45%, instructions at 60% of what a SIMD issues, LDS 21%:
// two waves a SIMD do not overlap them further.  Aggregate 248 to 284 us for two thirds of 1.3 GB
// (185 us at a copy's rate).  Heads of 64, packed: 712 to 770 us for 2.0 GB: latency of the
// chunk's steps at two waves a SIMD, and blocks that end late.  fp32: the fp32 matrix
// rate, a sixteenth of bf16's, busy 27 to 43%.
#pragma once

#include <atomic>
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

// Chunk length.  fp32 storage spends nothing on splitting the state, and gains by the
// smaller S.  (lin_output_kernel halves it where nk > nv.)
template <typename T>
constexpr int lin_steps() { return sizeof(T) == 4 ? 32 : 64; }
// Terms of an fp32 operand of a product: three of bf16 hold its 24 bits.
template <typename T> constexpr int lin_terms() { return sizeof(T) == 4 ? 1 : 3; }

// An operand of a product over 32 values of k: lane l holds row (or column)
// l % 16 and of lane group g = l / 16 the values k0 + 4 g + (0..3) in slots 0..3
// and k0 + 16 + 4 g + (0..3) in slots 4..7, as two 16x16 accumulator tiles have
// them.  (The instruction pairs equal slots.)
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
__device__ __forceinline__ void lin_mma(lin_f32x4 &acc, const LinFrag<bf16> &a, const LinFrag<bf16> &b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void lin_mma(lin_f32x4 &acc, const LinFrag<float> &a, const LinFrag<float> &b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], acc, 0, 0, 0);
}

// v as a sum of kTerms stored values, each the leading 8 bits of what is left: three
// hold the 24 bits of fp32.  Cut off, not rounded: a pair is packed by one
// instruction, and what is left is exact.  (v_dot2_f32_bf16 takes one instruction for it in
// place of two, but the output pass ran 815 us with it and 775 without.)  An
// infinity leaves NaN.
template <int kTerms>
__device__ __forceinline__ void lin_split(float (&v)[8], LinFrag<bf16> (&f)[kTerms]) {
#pragma unroll
    for (int n = 0; n < kTerms; ++n) {
        u32x4 h;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned a = __float_as_uint(v[2 * k]), b = __float_as_uint(v[2 * k + 1]);
            h[k] = __builtin_amdgcn_perm(b, a, 0x07060302);
            v[2 * k] -= __uint_as_float(a & 0xffff0000u);
            v[2 * k + 1] -= __uint_as_float(b & 0xffff0000u);
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

// Rows in LDS: granules of 16 bytes, kG to a row, without padding.  Granule c of
// a row lies at c ^ lin_pattern(row), so that what is read at once falls on
// different banks.  The pattern repeats after 16 rows, that of a | b is that of a ^ that
// of b for rows without a common bit, and what a lane chooses and what the step
// chooses are different bits of c: a read is one exclusive or with a constant away
// from its lane's base.
//   kLinNarrow  8 rows at two neighbouring granules (transposing reads for 16 columns)
//   kLinWide    4 rows at four neighbouring granules (for 32), and 32 rows at one
//   kLinFloat   rows 4 apart at four neighbouring granules; rows 0-3 and 12-15 at one
//               granule with rows 4-11 at its neighbour (lanes that a 16-byte read serves together)
enum LinOrder { kLinNarrow, kLinWide, kLinFloat };
template <int kG, LinOrder kOrder>
__device__ __forceinline__ constexpr int lin_pattern(int row) {
    constexpr int kLines = 16 / (kG < 16 ? kG : 16);  // rows that share 256 bytes
    if (kOrder == kLinFloat) return row & 15;
    if (kOrder == kLinWide) return (row / kLines & (kG / 4 - 1) & 3) << 2 | (row >> 2 & 3);
    const int up = (row & 3) | ((row >> 2 ^ row >> 3) & 1) << 2;
    return ((up / kLines) << 1 | (row >> 3 & 1)) & (kG - 1);
}

// fp32: the operand of the base's row, values k0 .. k0 + 31, k0 a multiple of 32;
// `t`: the tile, moved by a multiple of 16 rows.
template <int N>
struct LinRowReader {
    static constexpr int kG = N / 4;
    int base;  // granules
    __device__ __forceinline__ LinRowReader(int row, int g) : base(row * kG + (g ^ lin_pattern<kG, kLinFloat>(row))) {}
    __device__ __forceinline__ void operator()(LinFrag<float> &f, const u32x4 *t, int k0) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const u32x4 u = t[base ^ (k0 / 4 + 4 * k)];
            __builtin_memcpy(&f.v[4 * k], &u, 16);
        }
    }
};
// The operand of column c0 + 16 n + lane % 16, rows s0 .. s0 + 31; s0, c0
// multiples of 32.  bf16: two transposing LDS loads, in which, of 16 lanes, lane
// m addresses four columns of row m / 4 and lane i receives column i of the four
// rows.
template <typename T, int N>
struct LinColReader;
template <int N>
struct LinColReader<bf16, N> {
    static constexpr int kG = N / 8;
    int base;  // bytes
    __device__ __forceinline__ explicit LinColReader(int lane) {
        const int row = 4 * (lane >> 4) + ((lane & 15) >> 2);
        base = 16 * (row * kG + (((lane >> 1) & 1) ^ lin_pattern<kG, kLinNarrow>(row))) + 8 * (lane & 1);
    }
    __device__ __forceinline__ void operator()(LinFrag<bf16> &f, const u32x4 *t, int s0, int col) const {
        const char *p = reinterpret_cast<const char *>(t) + (base ^ 2 * col) + 16 * s0 * kG;
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lin_lds_i16x4 *)p));
        const u32x2 b =
            __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lin_lds_i16x4 *)(p + 16 * 16 * kG)));
        const u32x4 u = {a.x, a.y, b.x, b.y};
        f.v = __builtin_bit_cast(lin_bf16x8, u);
    }
};
template <int N>
struct LinColReader<float, N> {
    static constexpr int kG = N / 4;
    int base;  // values
    __device__ __forceinline__ explicit LinColReader(int lane) {
        const int g = lane >> 4, col = lane & 15;
        base = 4 * (4 * g * kG + (col / 4 ^ lin_pattern<kG, kLinFloat>(4 * g))) + col % 4;
    }
    __device__ __forceinline__ void operator()(LinFrag<float> &f, const u32x4 *t, int s0, int col) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // (of 16 rows, the pattern of 4 g + e is that of 4 g ^ that of e)
            const int row = s0 + e % 4 + 16 * (e / 4);
            f.v[e] = reinterpret_cast<const float *>(t)[(base ^ (col ^ 4 * lin_pattern<kG, kLinFloat>(e % 4))) + 4 * row * kG];
        }
    }
};

// A barrier for handing LDS between waves that does not wait for loads from
// memory in flight (__syncthreads does).
__device__ __forceinline__ void lin_barrier() {
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

// v, from here on unknown to the compiler: what is computed from it inside a loop
// (LDS addresses, mostly) is not kept in registers from round to round.
__device__ __forceinline__ int lin_afresh(int v) {
    __asm__ volatile("" : "+v"(v));
    return v;
}

// A chunk's rows of one tensor on their way through registers to LDS: granule
// i * kThreads + tid of the tile.
template <typename T, int N, int kC, int kThreads, LinOrder kOrder>
struct LinTile {
    static constexpr int kG = N * (int)sizeof(T) / 16, kCount = kC * kG / kThreads, kRows = kThreads / kG;
    static_assert(kC * kG % kThreads == 0 && kThreads % kG == 0, "whole granules per thread");
    u32x4 r[kCount];
    // `at`: the head's values of the chunk's first step; the next steps lie `dir`
    // times `stride` bytes (less than 2^22) further on; `width` bytes of a row are
    // the head's.  Rows past the end, and values past the width, lie outside the
    // descriptor and are read as zeros (offsets below it wrap around).
    __device__ __forceinline__ void load(const char *at, int32_t stride, int dir, int width, int rows) {
        const unsigned tid = lin_afresh(threadIdx.x);
        const int c = tid % kG * 16;
        const int32_t low = dir < 0 ? (rows - 1) * stride : 0;
        const __amdgpu_buffer_rsrc_t d = make_rsrc(at - low, (rows - 1) * stride + width);
        const unsigned to = c < width ? (unsigned)(__mul24((int)(tid / kG), dir * stride) + c + low) : 0x80000000u;
#pragma unroll
        for (int i = 0; i < kCount; ++i)
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(d, to + (unsigned)(i * kRows * dir * stride), 0, 0);
    }
    __device__ __forceinline__ void store(u32x4 *t) const {
        const unsigned tid = lin_afresh(threadIdx.x);
        const int at = tid ^ lin_pattern<kG, kOrder>(tid / kG);
        static_assert((kRows & (kRows - 1)) == 0, "a row's pattern is that of its bits below kRows ^ that of the others");
#pragma unroll
        for (int i = 0; i < kCount; ++i) t[(at ^ lin_pattern<kG, kOrder>(i * kRows % 16)) + i * kThreads] = r[i];
    }
};

// A value that every lane holds, in a scalar register.
__device__ __forceinline__ float lin_uniform(float v) { return __int_as_float(uniform(__float_as_int(v))); }
__device__ __forceinline__ int64_t lin_uniform(int64_t v) {
    return (int64_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v);
}

// Where a block works.
struct LinPlace {
    int64_t begin, end;  // steps of its sequence
    int64_t from, count; // its own, counted in the direction of the pass
    int64_t part;        // its entry of the parts' states
    int64_t index;       // its number in the sequence
    int row;             // sequence (or batch row)
    bool first, last;
};
__device__ __forceinline__ bool lin_place(const LinParams &p, int64_t part, LinPlace &me) {
    if (p.table) {
        const LinSeg s = p.table[part];
        if (s.index < 0) return false;
        me.begin = s.begin, me.end = s.end, me.row = s.seq, me.index = s.index, me.part = s.slot;
    } else {
        const int64_t per = p.segs / p.Bsz;
        me.row = (int)(part / per);
        me.index = part - me.row * per;
        me.begin = me.row * p.L, me.end = me.begin + p.L;
        me.part = part;
    }
    me.begin = lin_uniform(me.begin), me.end = lin_uniform(me.end), me.index = lin_uniform(me.index);
    me.part = lin_uniform(me.part);
    me.row = uniform(me.row);
    me.from = me.index * p.seg_len;
    const int64_t left = me.end - me.begin - me.from;
    me.count = left < p.seg_len ? left : p.seg_len;
    me.first = me.index == 0, me.last = left <= p.seg_len;
    return left > 0;
}

// Where a lane's values of a state lie whose element (row, column) is at row * sn +
// column * sc: column `col`, rows from `row` on; nk rows are there (a multiple of
// 8), and nv columns.
struct LinWhere {
    int32_t at, step;  // bytes: of the first value, from row to row
    int rows;          // of its column, from that value on
    __device__ __forceinline__ LinWhere(int sn, int sc, int nk, int nv, int col, int row)
        : at(4 * (col * sc + row * sn)), step(4 * sn), rows(col < nv ? nk - row : 0) {}
    __device__ __forceinline__ unsigned of(int row) const { return row < rows ? (unsigned)(at + row * step) : 0x80000000u; }
    // four rows of a state of `count` values
    __device__ __forceinline__ void load(lin_f32x4 &v, __amdgpu_buffer_rsrc_t d, int row) const {
        if (uniform(step) == 4) {
            v = __builtin_bit_cast(lin_f32x4, __builtin_amdgcn_raw_buffer_load_b128(d, of(row), 0, 0));
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(d, of(row + r), 0, 0));
        }
    }
    __device__ __forceinline__ void store(const lin_f32x4 &v, __amdgpu_buffer_rsrc_t d, int row) const {
        if (uniform(step) == 4) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), d, of(row), 0, 0);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[r]), d, of(row + r), 0, 0);
        }
    }
};
// A wave's columns of a state: register r of tile n of block i of lane (col, g)
// is row 32 i + 16 n + 4 g + r.
template <int NK>
struct LinState {
    lin_f32x4 h[NK / 32][2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NK / 32; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) h[i][0][r] = h[i][1][r] = 0.f;
    }
    __device__ __forceinline__ void load(const float *src, int64_t count, const LinWhere &w) {
        const __amdgpu_buffer_rsrc_t d = make_rsrc(src, (int32_t)count * 4);
#pragma unroll
        for (int i = 0; i < NK / 16; ++i) w.load(h[i / 2][i % 2], d, 16 * i);
    }
    __device__ __forceinline__ void store(float *dst, int64_t count, const LinWhere &w) const {
        const __amdgpu_buffer_rsrc_t d = make_rsrc(dst, (int32_t)count * 4);
#pragma unroll
        for (int i = 0; i < NK / 16; ++i) w.store(h[i / 2][i % 2], d, 16 * i);
    }
    __device__ __forceinline__ void fade(float factor, const LinState &add) {
        const lin_f32x4 f = {factor, factor, factor, factor};
#pragma unroll
        for (int i = 0; i < NK / 16; ++i) h[i / 2][i % 2] = __builtin_elementwise_fma(h[i / 2][i % 2], f, add.h[i / 2][i % 2]);
    }
};

// The same for tiles of 32 columns: register 8 j + e of tile i is row 32 i + 16 j +
// 8 g + e, and lane l % 32 stands for column lin_turn(l % 32).
template <int NK>
struct LinWideState {
    lin_f32x16 h[NK / 32];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NK / 32; ++i) h[i] = (lin_f32x16)(0.f);
    }
    template <typename F>
    static __device__ __forceinline__ void each(F f) {  // tile, register and row of each four
#pragma unroll
        for (int i = 0; i < NK / 8; ++i) f(i / 4, i % 4 * 4, 16 * (i / 2) + 4 * (i % 2));
    }
    __device__ __forceinline__ void load(const float *src, int64_t count, const LinWhere &w) {
        const __amdgpu_buffer_rsrc_t d = make_rsrc(src, (int32_t)count * 4);
        each([&](int i, int r, int row) {
            lin_f32x4 v;
            w.load(v, d, row);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[i][r + e] = v[e];
        });
    }
    __device__ __forceinline__ void store(float *dst, int64_t count, const LinWhere &w) const {
        const __amdgpu_buffer_rsrc_t d = make_rsrc(dst, (int32_t)count * 4);
        each([&](int i, int r, int row) { w.store(lin_f32x4{h[i][r], h[i][r + 1], h[i][r + 2], h[i][r + 3]}, d, row); });
    }
    __device__ __forceinline__ void fade(float factor, const LinWideState &add) {
#pragma unroll
        for (int i = 0; i < NK / 32; ++i) h[i] = __builtin_elementwise_fma(h[i], (lin_f32x16)(factor), add.h[i]);
    }
};

// The state that enters the output pass's part: the carried one, or what the few
// parts before it add, of seg_len steps each.  `there`, `outside`: the
// lane's place in `states` and in h_init.
template <typename State>
__device__ __forceinline__ void lin_enter(State &hs, const LinParams &p, const LinPlace &me, int h, const LinWhere &there,
                                          const LinWhere &outside) {
    const int64_t state = (int64_t)p.nk * p.nv;
    const float *sum = p.states + (me.part * p.H + h) * state;
    if (!me.first && me.end - me.begin > kLinDirect * p.seg_len) {
        hs.load(sum, state, there);
        return;
    }
    if (p.states && p.copy_first)
        hs.load(sum - me.index * p.H * state, state, there);
    else if (p.h_init)
        hs.load(p.h_init + ((int64_t)me.row * p.H + h) * state, state, outside);
    const float fade = (float)exp((double)p.log_decay[h] * (double)p.seg_len);
    for (int64_t i = me.index - 1; i >= 0; --i) {
        State add;
        add.load(sum - i * p.H * state, state, there);
        hs.fade(fade, add);
    }
}

// The log decay in base-2 units.  Below -1e4 every power but the 0th is 0
// (and 0 times it stays 0: a = -inf is a state without memory).
__device__ __forceinline__ float lin_log2_decay(float a) {
    const float a2 = a * kLog2e;
    return a2 < -1e4f ? -1e4f : a2;
}

// The factors that the state fades by, chunk after chunk.  A factor near 1 that
// is always rounded to fp32 the same way would be off by the same 2^-25 at every
// chunk of a long memory; here each factor makes up for what the ones before it
// were off by.
struct LinFading {
    double exact, inverse, error;
    __device__ __forceinline__ void set(double factor) {
        exact = factor;
        inverse = factor > 1e-30 ? 1.0 / factor : 0.0;
        error = 0.0;
        scalars(exact, inverse);
    }
    __device__ __forceinline__ float next() {
        const double now = fma_(exact, error, exact);
        const float f = (float)now;
        error = (now - (double)f) * inverse;
        scalars(error, error);
        return lin_uniform(f);
    }
    // (the same in every lane: held in scalar registers)
    static __device__ __forceinline__ void scalars(double &a, double &b) {
        a = __hiloint2double(uniform(__double2hiint(a)), uniform(__double2loint(a)));
        b = __hiloint2double(uniform(__double2hiint(b)), uniform(__double2loint(b)));
    }
};

// Waves of a SIMD that the registers are cut for: what the chunk in LDS leaves room
// for, and with more registers where few waves stage wide rows.
template <typename T, int NK, int NV>
constexpr int lin_waves() { return sizeof(T) == 4 || NK > NV ? 3 : 4; }

// kOutput (fp32 storage): y of every step, and the last part's state to h_final.
// Otherwise the state that a part adds (from zero) to the next part's entry of `states`, each
// step weighted by its distance from the part's end.
template <typename T, int NK, int NV, LinPass kPass>
__global__ __launch_bounds__(4 * NV, (lin_waves<T, NK, NV>())) void lin_chunk_kernel(LinParams p) {
    constexpr int kC = lin_steps<T>(), kTT = kC / 16, kJ = kC / 32, kThreads = 4 * NV;
    constexpr int kRow = NK == 96 ? 128 : NK;  // values of a row in LDS
    constexpr int kGK = kRow * (int)sizeof(T) / 16, kGV = NV * (int)sizeof(T) / 16;
    constexpr bool kOut = kPass == LinPass::kOutput;
    static_assert(!kOut || sizeof(T) == 4, "bf16 storage: lin_output_kernel");
    constexpr int kTerms = lin_terms<T>();
    constexpr int kFragWords = (int)sizeof(LinFrag<T>) / 16;  // 16-byte words of a fragment
    __shared__ __attribute__((aligned(16))) u32x4 lq[kOut ? kC * kGK : 1];
    __shared__ __attribute__((aligned(16))) u32x4 lk[kC * kGK];
    __shared__ __attribute__((aligned(16))) u32x4 lv[kC * kGV];
    __shared__ __attribute__((aligned(16))) u32x4 ls[kOut ? kTT * kFragWords * kWave : 1];  // 32 steps s of 16 steps t
    __shared__ __attribute__((aligned(16))) float lw[kC];
    __shared__ float lp[kOut ? kC + 31 : 1];

    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const int g = lane >> 4, li = lane & 15;
    const int block = p.first + xcd_remap(blockIdx.x, gridDim.x);
    const int h = block % p.H;
    LinPlace me;
    if (!lin_place(p, block / p.H, me)) return;
    if (!kOut && me.last) return;

    const float a2 = lin_uniform(lin_log2_decay(p.log_decay[h]));
    const int off = p.reverse ? 0 : 1;  // decays of an entering state at its first step
    const int col = 16 * wave + li;
    const int64_t state = (int64_t)p.nk * p.nv;

    LinState<NK> hs;
    hs.zero();
    if constexpr (kOut) {
        lin_enter(hs, p, me, h, LinWhere(p.tn, p.tc, p.nk, p.nv, col, 4 * g), LinWhere(p.sn, p.sc, p.nk, p.nv, col, 4 * g));
    }

    // ---- the tensors' rows, chunk after chunk
    const int32_t es = sizeof(T), ys = 4;
    const int32_t q_step = (p.H / p.gq) * p.nk * es, k_step = (p.H / p.gk) * p.nk * es, v_step = (p.H / p.gv) * p.nv * es;
    const int32_t y_step = p.H * p.nv * ys;
    const int chunks = (int)((me.count + kC - 1) / kC), tail = (int)(me.count - (int64_t)(chunks - 1) * kC);
    const int dir = p.reverse ? -1 : 1;
    const int64_t from = p.reverse ? me.end - 1 - me.from : me.begin + me.from;
    const char *qp = static_cast<const char *>(p.q) + from * q_step + (h / p.gq) * p.nk * es;
    const char *kp = static_cast<const char *>(p.k) + from * k_step + (h / p.gk) * p.nk * es;
    const char *vp = static_cast<const char *>(p.v) + from * v_step + (h / p.gv) * p.nv * es;
    char *yp = static_cast<char *>(p.y) + from * y_step + h * p.nv * ys;
    constexpr LinOrder kOrder = sizeof(T) == 4 ? kLinFloat : kLinNarrow;
    LinTile<T, kRow, kC, kThreads, kOrder> tq, tk;
    LinTile<T, NV, kC, kThreads, kOrder> tv;
    auto fetch = [&](int rows) {  // the next chunk's
        if constexpr (kOut) tq.load(qp, q_step, dir, p.nk * es, rows), qp += (int64_t)dir * kC * q_step;
        tk.load(kp, k_step, dir, p.nk * es, rows), kp += (int64_t)dir * kC * k_step;
        tv.load(vp, v_step, dir, p.nv * es, rows), vp += (int64_t)dir * kC * v_step;
    };
    // the staged rows to LDS, and the weights of the chunk's rows in a state
    // `left` steps behind its first (rows past the end are zeros)
    auto place = [&](int left, bool weights) {
        if constexpr (kOut) tq.store(lq);
        tk.store(lk);
        tv.store(lv);
        if (weights && threadIdx.x < kC) {
            const int back = left - off - (int)threadIdx.x;
            lw[threadIdx.x] = back >= 0 ? fast_exp2((float)back * a2) * p.k_scale : 0.f;
        }
    };

    // ---- weights L^n of S at lp[n + 31], 0 for n < 0, and L^16
    const float fade16 = lin_uniform(fast_exp2(16.f * a2));
    if constexpr (kOut) {
        if (threadIdx.x < kC + 31) {
            const int n = (int)threadIdx.x - 31;
            lp[threadIdx.x] = n >= 0 ? fast_exp2((float)n * a2) * (p.y_scale * p.k_scale) : 0.f;
        }
    }

    // One chunk of `rows` steps, its rows in LDS; kMore: another one follows, of `next`
    // rows, `left` steps before the end; kIdle: the wave's columns are not there, it only
    // moves rows and forms S (heads of 72 in fp32, 2 x 8192 steps of 32: 318 -> 267 us).
    auto chunk = [&](auto idle, auto more, int rows, int next, int left, float decay) {
        constexpr bool kIdle = decltype(idle)::value, kMore = decltype(more)::value;
        if constexpr (kMore) fetch(next);
        lin_f32x4 y[kOut ? kTT : 1];
        if constexpr (kOut) {
            // ---- S^T = k q^T (rows s, columns t), weighted, to LDS as operands: a wave per 16 steps t
            if (wave < kTT) {
                const int l = lin_afresh(threadIdx.x) & (kWave - 1), g = l >> 4, li = l & 15;
                lin_f32x4 s[2];
#pragma unroll
                for (int r = 0; r < 4; ++r) s[0][r] = s[1][r] = 0.f;
                const LinRowReader<kRow> row(li, g);
                LinFrag<T> f3[2][3];  // the next step's operands are read ahead
                auto ahead = [&](int k0) {
                    LinFrag<T>(&f)[3] = f3[k0 / 32 % 2];
                    row(f[0], lq + 16 * wave * kGK, k0);
                    row(f[1], lk, k0);
                    row(f[2], lk + 16 * kGK, k0);
                };
                ahead(0);
#pragma unroll
                for (int k0 = 0; k0 < NK; k0 += 32) {
                    const LinFrag<T>(&f)[3] = f3[k0 / 32 % 2];
                    if (k0 + 32 < NK) ahead(k0 + 32);
                    lin_mma(s[0], f[1], f[0]);
                    lin_mma(s[1], f[2], f[0]);
                    __builtin_amdgcn_sched_barrier(0);  // (operands read further ahead would not fit in registers)
                }
                // weights by how far s is back from t; above the diagonal 0, whatever S is there
                const int diag = 16 * wave + li - 4 * g;
                const float *weight = lp + 31 + diag;
                LinFrag<T> w;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = 16 * (e / 4) + e % 4;
                    const float v = s[e / 4][e % 4] * weight[-at];
                    w.v[e] = at <= diag ? v : 0.f;
                }
                u32x4 u[kFragWords];
                __builtin_memcpy(u, &w, sizeof u);
#pragma unroll
                for (int k = 0; k < kFragWords; ++k) ls[(wave * kFragWords + k) * kWave + l] = u[k];
            }
            // ---- y^T = H q^T (rows of v's columns, columns t); the state fades on the way
            if constexpr (!kIdle) {
                const int l = lin_afresh(threadIdx.x) & (kWave - 1);
                const LinRowReader<kRow> q_row(l & 15, l >> 4);
#pragma unroll
                for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[tt][r] = 0.f;
                LinFrag<T> qf[2][kTT];
                auto ahead = [&](int i) {
#pragma unroll
                    for (int tt = 0; tt < kTT; ++tt) q_row(qf[i % 2][tt], lq + 16 * tt * kGK, 32 * i);
                };
                ahead(0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < NK / 32; ++i) {
                    const lin_f32x4 h0 = hs.h[i][0], h1 = hs.h[i][1];
                    LinFrag<T> hf;
#pragma unroll
                    for (int e = 0; e < 8; ++e) hf.v[e] = e < 4 ? h0[e % 4] : h1[e % 4];
                    hs.h[i][0] = h0 * decay, hs.h[i][1] = h1 * decay;
                    if (i + 1 < NK / 32) ahead(i + 1);
#pragma unroll
                    for (int tt = 0; tt < kTT; ++tt) lin_mma(y[tt], hf, qf[i % 2][tt]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if constexpr (!kIdle) {
                // L^{t + off}
                float f = fast_exp2((float)((lin_afresh(threadIdx.x) & 15) + off) * a2) * p.y_scale;
#pragma unroll
                for (int tt = 0; tt < kTT; ++tt) {
                    y[tt] *= f;
                    f *= fade16;
                }
            }
        }
        // ---- H += weighted v k^T
        LinFrag<T> vf[kJ];
        if constexpr (!kIdle) {
            const int l = lin_afresh(threadIdx.x) & (kWave - 1);
            const LinColReader<T, NV> v_col(l);
            const LinColReader<T, kRow> k_col(l);
            const float *weight = lw + 4 * (l >> 4);
            constexpr int kI = NK / 32;
            LinFrag<T> kf[2][2];
            auto ahead = [&](int at) {  // k's rows 32 j, columns 32 i for at = j kI + i
                k_col(kf[at % 2][0], lk, 32 * (at / kI), 32 * (at % kI));
                k_col(kf[at % 2][1], lk, 32 * (at / kI), 32 * (at % kI) + 16);
            };
            v_col(vf[0], lv, 0, 16 * wave);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                auto weighted = [&](auto &wf) {
                    float w[8];
                    const lin_f32x4 a = *reinterpret_cast<const lin_f32x4 *>(weight + 32 * j);
                    const lin_f32x4 b = *reinterpret_cast<const lin_f32x4 *>(weight + 32 * j + 16);
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = lin_elem(vf[j], e) * (e < 4 ? a[e % 4] : b[e % 4]);
                    lin_split(w, wf);
                };
                LinFrag<T> wf[kTerms];
                weighted(wf);
                if (j == 0) {
                    __builtin_amdgcn_sched_barrier(0);
                    ahead(0);
                }
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                    const int at = j * kI + i;
                    if (at + 1 < kJ * kI) ahead(at + 1);
                    if (i + 1 == kI && j + 1 < kJ) v_col(vf[j + 1], lv, 32 * (j + 1), 16 * wave);
#pragma unroll
                    for (int n = 0; n < kTerms; ++n) {
                        lin_mma(hs.h[i][0], kf[at % 2][0], wf[n]);
                        lin_mma(hs.h[i][1], kf[at % 2][1], wf[n]);
                    }
                    if constexpr (kOut) __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        lin_barrier();  // S is written; every wave is done with the chunk's rows
        if constexpr (kMore) place(kOut ? next : left, !kOut || next != kC);
        if constexpr (kOut && !kIdle) {
            // ---- y^T += v^T S^T
            const int l = lin_afresh(threadIdx.x) & (kWave - 1), g = l >> 4, li = l & 15;
#pragma unroll
            for (int tt = 0; tt < kTT; ++tt) {
                u32x4 u[kFragWords];
#pragma unroll
                for (int k = 0; k < kFragWords; ++k) u[k] = ls[(tt * kFragWords + k) * kWave + l];
                LinFrag<T> f;
                __builtin_memcpy(&f, u, sizeof u);
                lin_mma(y[tt], vf[0], f);
            }
            // ---- y out: 4 consecutive values of a step per lane
            const int at = 16 * wave + 4 * g;
            const int32_t low = dir < 0 ? (rows - 1) * y_step : 0;
            const __amdgpu_buffer_rsrc_t d = make_rsrc(yp - low, (rows - 1) * y_step + p.nv * ys);
            const unsigned to = at < p.nv ? (unsigned)(__mul24(li, dir * y_step) + at * ys + low) : 0x80000000u;
#pragma unroll
            for (int tt = 0; tt < kTT; ++tt)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[tt]), d,
                                                       to + (unsigned)(16 * tt * dir * y_step), 0, 0);
            yp += (int64_t)dir * kC * y_step;
        }
        if constexpr (kMore) lin_barrier();  // the next chunk's rows are in, S is read
    };
    const int first = chunks > 1 ? kC : tail;
    const LinWhere outside(p.sn, p.sc, p.nk, p.nv, col, 4 * g), there(1, p.nk, p.nk, p.nv, col, 4 * g);
    fetch(first);
    place(kOut ? first : (int)me.count, true);
    lin_barrier();
    auto run = [&](auto idle) {
        if constexpr (kOut) {
            LinFading fading;
            fading.set(exp((double)p.log_decay[h] * kC));
            for (int c = chunks; c > 1; --c) chunk(idle, std::true_type{}, kC, c > 2 ? kC : tail, 0, fading.next());
            chunk(idle, std::false_type{}, tail, 0, 0, (float)exp((double)p.log_decay[h] * tail));
            if (!idle() && me.last && p.h_final != nullptr)
                hs.store(p.h_final + ((int64_t)me.row * p.H + h) * state, state, outside);
        } else {  // (never a sequence's last part: whole chunks)
            int left = (int)me.count;
            for (int c = chunks; c > 1; --c) chunk(idle, std::true_type{}, kC, kC, left -= kC, 0.f);
            chunk(idle, std::false_type{}, kC, 0, 0, 0.f);
            if (!idle()) hs.store(p.states + ((me.part + 1) * p.H + h) * state, state, there);
        }
    };
    if (16 * wave < p.nv) run(std::false_type{});
    else run(std::true_type{});
}

// A SIMD serves its oldest wave first, so of two blocks on a compute unit the one that
// came first runs ahead and the other one's last chunks have the unit to
// themselves, at two thirds of its rate (2 x 64 chunks, two terms: they ended after 415 and
// 525 us).  With the later block's waves at the higher priority, the first one's in
// every other chunk, both end together (after 460 to 500 us).  Later waves are
// known by their slot, of which the first wave of a SIMD has number 0; once blocks
// follow each other the order is by chance, and so is who waits.
__device__ __forceinline__ bool lin_came_later() {
    return (__builtin_amdgcn_s_getreg(4 | 3 << 11) & 15) != 0;  // HW_ID's wave slot
}
__device__ __forceinline__ void lin_take_turns(bool later, int chunk) {
    if (later || chunk % 2) __builtin_amdgcn_s_setprio(1);
    else __builtin_amdgcn_s_setprio(0);
}

// ---- bf16's output pass: tiles of 32x32 (v_mfma_f32_32x32x16_bf16), a wave per 32
// columns of v.  The operands of a product over 16 values of k: lane l holds row
// l % 32, values k0 + 8 (l / 32) + (0..7).  A product's rows that lane l % 32 stands for
// are turned, so that registers 8 j + e of its result are rows 16 j + 8 (l / 32) + e:
// 8 of them are the next product's operand in place.
__device__ __forceinline__ constexpr int lin_turn(int l) { return (l & 0x13) | (l & 4) << 1 | (l & 8) >> 1; }
__device__ __forceinline__ void lin_mma_wide(lin_f32x16 &acc, const LinFrag<bf16> &a, const LinFrag<bf16> &b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}
// Row `row` at values k0 .. k0 + 15, k0 a multiple of 16; `t`: the tile, moved by
// a multiple of 32 rows.
template <int N>
struct LinWideRow {
    static constexpr int kG = N / 8;
    int base;
    __device__ __forceinline__ LinWideRow(int row, int g) : base(row * kG + (g ^ lin_pattern<kG, kLinWide>(row))) {}
    __device__ __forceinline__ void operator()(LinFrag<bf16> &f, const u32x4 *t, int k0) const {
        f.v = __builtin_bit_cast(lin_bf16x8, t[base ^ k0 / 8]);
    }
};
// Column c0 + lin_turn(lane % 32) at rows s0 .. s0 + 15; s0 a multiple of 16, c0 of 32.
template <int N>
struct LinWideCol {
    static constexpr int kG = N / 8;
    int base;  // bytes
    __device__ __forceinline__ explicit LinWideCol(int lane) {
        const int row = 8 * (lane >> 5) + ((lane & 15) >> 2), c = 2 * (lane >> 4 & 1) + (lane & 1);
        base = 16 * (row * kG + (c ^ lin_pattern<kG, kLinWide>(row))) + 8 * (lane >> 1 & 1);
    }
    __device__ __forceinline__ void operator()(LinFrag<bf16> &f, const u32x4 *t, int s0, int c0) const {
        // (4 rows on, the pattern differs by that of row 4)
        const char *p = reinterpret_cast<const char *>(t) + 16 * s0 * kG;
        const char *a = p + (base ^ 2 * c0), *b = p + (base ^ (2 * c0 ^ 16 * lin_pattern<kG, kLinWide>(4))) + 16 * 4 * kG;
        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lin_lds_i16x4 *)a));
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lin_lds_i16x4 *)b));
        const u32x4 u = {x.x, x.y, y.x, y.y};
        f.v = __builtin_bit_cast(lin_bf16x8, u);
    }
};

template <int NK, int NV>
__global__ __launch_bounds__(2 * NV, 2) void lin_output_kernel(LinParams p) {
    typedef bf16 T;
    // Half the steps where the registers of few waves would stage wide rows.
    constexpr int kC = NK > NV ? 32 : 64, kTT = kC / 32, kThreads = 2 * NV, kWaves = NV / 32;
    constexpr int kRow = NK == 96 ? 128 : NK;  // values of a row in LDS
    constexpr int kGK = kRow / 8, kGV = NV / 8, kTerms = lin_terms<T>();
    constexpr int kTiles = kTT == 2 ? 3 : 1;  // tiles of S with s <= t: steps s, t from (0, 0), (0, 32), (32, 32)
    __shared__ __attribute__((aligned(16))) u32x4 lq[kC * kGK];
    __shared__ __attribute__((aligned(16))) u32x4 lk[kC * kGK];
    __shared__ __attribute__((aligned(16))) u32x4 lv[kC * kGV];
    // S as operands: steps s of the halves j of every tile.  The second half of a tile on the
    // diagonal is 0 for the tile's first 16 steps t, and only the others are kept (heads of 64:
    // four blocks on a compute unit instead of three, 845 -> 735 us for 65536 packed steps of 80 heads).
    constexpr int kDiagonals = kTT;
    __shared__ __attribute__((aligned(16))) u32x4 ls[(2 * kTiles * kWave - kDiagonals * kWave / 2) * kTerms];
    auto s_at = [](int tile, int j, int term, int l) {  // where lane l's operand lies
        if (tile % 2 == 0 && j == 1)
            return ((2 * kTiles - kDiagonals) * kTerms * 2 + tile / 2 * kTerms + term) * (kWave / 2) + (l >> 5) * 16 + (l & 15);
        return ((tile == 0 ? 0 : tile == 1 ? 1 + j : 3) * kTerms + term) * kWave + l;
    };
    __shared__ __attribute__((aligned(16))) float lw[kC];
    __shared__ float lp[kC + 31];

    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const int g = lane >> 5, li = lane & 31;
    const int block = p.first + xcd_remap(blockIdx.x, gridDim.x);
    const int h = block % p.H;
    LinPlace me;
    if (!lin_place(p, block / p.H, me)) return;

    const float a2 = lin_uniform(lin_log2_decay(p.log_decay[h]));
    const int off = p.reverse ? 0 : 1;  // decays of an entering state at its first step
    const int col = 32 * wave + lin_turn(li);

    LinWideState<NK> hs;
    hs.zero();
    lin_enter(hs, p, me, h, LinWhere(p.tn, p.tc, p.nk, p.nv, col, 8 * g), LinWhere(p.sn, p.sc, p.nk, p.nv, col, 8 * g));

    // ---- the tensors' rows, chunk after chunk
    const int32_t es = sizeof(T), ys = p.y_f32 ? 4 : 2;
    const int32_t q_step = (p.H / p.gq) * p.nk * es, k_step = (p.H / p.gk) * p.nk * es, v_step = (p.H / p.gv) * p.nv * es;
    const int32_t y_step = p.H * p.nv * ys;
    const int chunks = (int)((me.count + kC - 1) / kC), tail = (int)(me.count - (int64_t)(chunks - 1) * kC);
    const int dir = p.reverse ? -1 : 1;
    const int64_t from = p.reverse ? me.end - 1 - me.from : me.begin + me.from;
    const char *qp = static_cast<const char *>(p.q) + from * q_step + (h / p.gq) * p.nk * es;
    const char *kp = static_cast<const char *>(p.k) + from * k_step + (h / p.gk) * p.nk * es;
    const char *vp = static_cast<const char *>(p.v) + from * v_step + (h / p.gv) * p.nv * es;
    char *yp = static_cast<char *>(p.y) + from * y_step + h * p.nv * ys;
    LinTile<T, kRow, kC, kThreads, kLinWide> tq, tk;
    LinTile<T, NV, kC, kThreads, kLinWide> tv;
    auto fetch = [&](int rows) {  // the next chunk's
        tq.load(qp, q_step, dir, p.nk * es, rows), qp += (int64_t)dir * kC * q_step;
        tk.load(kp, k_step, dir, p.nk * es, rows), kp += (int64_t)dir * kC * k_step;
        tv.load(vp, v_step, dir, p.nv * es, rows), vp += (int64_t)dir * kC * v_step;
    };
    // the staged rows to LDS, and the weights of the chunk's rows in the state at its end
    // (rows past it are zeros)
    auto place = [&](int rows, bool weights) {
        tq.store(lq);
        tk.store(lk);
        tv.store(lv);
        if (weights && threadIdx.x < kC) {
            const int back = rows - off - (int)threadIdx.x;
            lw[threadIdx.x] = back >= 0 ? fast_exp2((float)back * a2) * p.k_scale : 0.f;
        }
    };

    // ---- weights L^n of S at lp[n + 31], 0 for n < 0, and L^{t + off} of this lane's steps
    if (threadIdx.x < kC + 31) {
        const int n = (int)threadIdx.x - 31;
        lp[threadIdx.x] = n >= 0 ? fast_exp2((float)n * a2) * (p.y_scale * p.k_scale) : 0.f;
    }
    float fade[kTT];
#pragma unroll
    for (int tt = 0; tt < kTT; ++tt) fade[tt] = fast_exp2((float)(32 * tt + li + off) * a2) * p.y_scale;

    // One chunk, its rows in LDS; kMore: another one follows, of `next` rows; kIdle: as above.
    auto chunk = [&](auto idle, auto more, int rows, int next, float decay) {
        constexpr bool kIdle = decltype(idle)::value, kMore = decltype(more)::value;
        if constexpr (kMore) fetch(next);
        // ---- S^T = k q^T (rows s, columns t), weighted, to LDS as operands
#pragma unroll
        for (int tile = 0; tile < kTiles; ++tile) {
            // (of two waves, one takes the tile below the diagonal)
            if (kWaves >= 4 || kTiles == 1 ? wave != tile : (wave == 1) != (tile == 1)) continue;
            const int st = tile / 2, tt = (tile + 1) / 2;
            const int l = lin_afresh(threadIdx.x) & (kWave - 1), g = l >> 5, li = l & 31;
            lin_f32x16 s = (lin_f32x16)(0.f);
            const LinWideRow<kRow> q_row(li, g), k_row(lin_turn(li), g);
            LinFrag<T> f[3][2];  // operands of the step and the two after it
            auto ahead = [&](int k0) {
                q_row(f[k0 / 16 % 3][0], lq + 32 * tt * kGK, k0);
                k_row(f[k0 / 16 % 3][1], lk + 32 * st * kGK, k0);
            };
            ahead(0);
            ahead(16);
#pragma unroll
            for (int k0 = 0; k0 < NK; k0 += 16) {
                if (k0 + 32 < NK) ahead(k0 + 32);
                lin_mma_wide(s, f[k0 / 16 % 3][1], f[k0 / 16 % 3][0]);
                __builtin_amdgcn_sched_barrier(0);
            }
            // weights by how far s is back from t; above the diagonal 0, whatever S is there
            const int diag = 32 * tt + li - 32 * st - 8 * g;
            const float *weight = lp + 31 + diag;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float w[8];
                LinFrag<T> terms[kTerms];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = 16 * j + e;
                    const float v = s[8 * j + e] * weight[-at];
                    w[e] = st != tt || at <= diag ? v : 0.f;
                }
                lin_split<kTerms>(w, terms);
                if (st != tt || j == 0 || li >= 16)
#pragma unroll
                    for (int n = 0; n < kTerms; ++n) ls[s_at(tile, j, n, l)] = __builtin_bit_cast(u32x4, terms[n].v);
            }
        }
        lin_f32x16 y[kTT];
#pragma unroll
        for (int tt = 0; tt < kTT; ++tt) y[tt] = (lin_f32x16)(0.f);
        LinFrag<T> vf[kC / 16];
        if constexpr (!kIdle) {
            // ---- y^T = H q^T (rows of v's columns, columns t); the state fades on the way
            {
                const int l = lin_afresh(threadIdx.x) & (kWave - 1);
                const LinWideRow<kRow> q_row(l & 31, l >> 5);
                LinFrag<T> qf[3][kTT];
                auto ahead = [&](int k0) {
#pragma unroll
                    for (int tt = 0; tt < kTT; ++tt) q_row(qf[k0 / 16 % 3][tt], lq + 32 * tt * kGK, k0);
                };
                ahead(0);
                ahead(16);
#pragma unroll
                for (int k0 = 0; k0 < NK; k0 += 16) {
                    LinFrag<T> hf[kTerms];
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = hs.h[k0 / 32][k0 % 32 / 2 + e];
                    lin_split<kTerms>(v, hf);
                    if (k0 % 32) hs.h[k0 / 32] *= decay;
                    if (k0 + 32 < NK) ahead(k0 + 32);
#pragma unroll
                    for (int n = 0; n < kTerms; ++n)
#pragma unroll
                        for (int tt = 0; tt < kTT; ++tt) lin_mma_wide(y[tt], hf[n], qf[k0 / 16 % 3][tt]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int tt = 0; tt < kTT; ++tt) y[tt] *= fade[tt];
            // ---- H += weighted v k^T
            {
                const int l = lin_afresh(threadIdx.x) & (kWave - 1);
                const LinWideCol<NV> v_col(l);
                const LinWideCol<kRow> k_col(l);
                const float *weight = lw + 8 * (l >> 5);
                constexpr int kI = NK / 32, kAll = kC / 16 * kI;
                LinFrag<T> kf[3];
                auto ahead = [&](int at) { k_col(kf[at % 3], lk, 16 * (at / kI), 32 * (at % kI)); };  // k's rows 16 (at / kI)
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) v_col(vf[j], lv, 16 * j, 32 * wave);
                ahead(0);
                ahead(1);
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) {
                    float w[8];
                    const lin_f32x4 a = *reinterpret_cast<const lin_f32x4 *>(weight + 16 * j);
                    const lin_f32x4 b = *reinterpret_cast<const lin_f32x4 *>(weight + 16 * j + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = lin_elem(vf[j], e) * (e < 4 ? a[e % 4] : b[e % 4]);
                    LinFrag<T> wf[kTerms];
                    lin_split<kTerms>(w, wf);
#pragma unroll
                    for (int i = 0; i < kI; ++i) {
                        const int at = j * kI + i;
                        if (at + 2 < kAll) ahead(at + 2);
#pragma unroll
                        for (int n = 0; n < kTerms; ++n) lin_mma_wide(hs.h[i], kf[at % 3], wf[n]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        }
        lin_barrier();  // S is written; every wave is done with the chunk's rows
        if constexpr (kMore) place(next, next != kC);
        // ---- y^T += v^T S^T
        if constexpr (!kIdle) {
            const int l = lin_afresh(threadIdx.x) & (kWave - 1), g = l >> 5, li = l & 31;
#pragma unroll
            for (int n = 0; n < kTerms; ++n)
#pragma unroll
                for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        u32x4 u = ls[s_at(tile, j, n, l)];
                        if (tile % 2 == 0 && j == 1 && li < 16) u = u32x4{0, 0, 0, 0};
                        LinFrag<T> f;
                        f.v = __builtin_bit_cast(lin_bf16x8, u);
                        lin_mma_wide(y[(tile + 1) / 2], vf[2 * (tile / 2) + j], f);
                    }
            // ---- y out: 8 consecutive values of a step per lane
            const int32_t low = dir < 0 ? (rows - 1) * y_step : 0;
            const __amdgpu_buffer_rsrc_t d = make_rsrc(yp - low, (rows - 1) * y_step + p.nv * ys);
            const int32_t to0 = __mul24(li, dir * y_step) + low;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = 32 * wave + 16 * j + 8 * g;
                const unsigned to = at < p.nv ? (unsigned)(to0 + at * ys) : 0x80000000u;
#pragma unroll
                for (int tt = 0; tt < kTT; ++tt) {
                    const unsigned there = to + (unsigned)(32 * tt * dir * y_step);
                    if (p.y_f32) {
                        u32x4 a, b;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[e] = __float_as_uint(y[tt][8 * j + e]), b[e] = __float_as_uint(y[tt][8 * j + 4 + e]);
                        __builtin_amdgcn_raw_buffer_store_b128(a, d, there, 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b128(b, d, there + 16, 0, 0);
                    } else {
                        u32x4 u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const lin_f32x2 v = {y[tt][8 * j + 2 * e], y[tt][8 * j + 2 * e + 1]};
                            u[e] = __builtin_bit_cast(unsigned, __builtin_convertvector(v, lin_bf16x2));
                        }
                        __builtin_amdgcn_raw_buffer_store_b128(u, d, there, 0, 0);
                    }
                }
            }
            yp += (int64_t)dir * kC * y_step;
        }
        if constexpr (kMore) lin_barrier();  // the next chunk's rows are in, S is read
    };
    const int first = chunks > 1 ? kC : tail;
    fetch(first);
    place(first, true);
    lin_barrier();
    auto run = [&](auto idle) {
        LinFading fading;
        fading.set(exp((double)p.log_decay[h] * kC));
        const bool later = lin_came_later();
        for (int c = chunks; c > 1; --c) {
            lin_take_turns(later, c);
            chunk(idle, std::true_type{}, kC, c > 2 ? kC : tail, fading.next());
        }
        chunk(idle, std::false_type{}, tail, 0, (float)exp((double)p.log_decay[h] * tail));
        if (!idle() && me.last && p.h_final != nullptr) {
            const int64_t state = (int64_t)p.nk * p.nv;
            hs.store(p.h_final + ((int64_t)me.row * p.H + h) * state, state,
                     LinWhere(p.sn, p.sc, p.nk, p.nv, col, 8 * g));
        }
    };
    if (32 * wave < p.nv) run(std::false_type{});
    else run(std::true_type{});
}

template <typename T, int NK, int NV>
hipError_t lin_pass_n(LinPass pass, LinParams p, hipStream_t s) {
    const int64_t blocks = p.segs * p.H;
    constexpr int64_t kMost = 1 << 22;  // blocks of a launch (its threads stay below 2^32)
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < blocks && e == hipSuccess; first += kMost) {
        const dim3 grid((unsigned)(blocks - first < kMost ? blocks - first : kMost)), block(4 * NV);
        p.first = (int)first;
        if (pass == LinPass::kAggregate)
            hipLaunchKernelGGL((lin_chunk_kernel<T, NK, NV, LinPass::kAggregate>), grid, block, 0, s, p);
        else if constexpr (sizeof(T) == 2)
            hipLaunchKernelGGL((lin_output_kernel<NK, NV>), grid, dim3(2 * NV), 0, s, p);
        else
            hipLaunchKernelGGL((lin_chunk_kernel<T, NK, NV, LinPass::kOutput>), grid, block, 0, s, p);
        e = hipGetLastError();
    }
    return e;
}

// The kernels by head sizes: f(integral_constant NK, integral_constant NV).
template <typename F>
auto lin_sizes(int64_t nk, int64_t nv, F &&f) {
    using N64 = std::integral_constant<int, 64>;
    using N96 = std::integral_constant<int, 96>;
    using N128 = std::integral_constant<int, 128>;
    if (nv <= 64) return nk <= 64 ? f(N64{}, N64{}) : nk <= 96 ? f(N96{}, N64{}) : f(N128{}, N64{});
    return nk <= 64 ? f(N64{}, N128{}) : nk <= 96 ? f(N96{}, N128{}) : f(N128{}, N128{});
}

template <typename T>
hipError_t lin_pass_t(LinPass pass, const LinParams &p, hipStream_t s) {
    return lin_sizes(p.nk, p.nv, [&](auto nk, auto nv) { return lin_pass_n<T, nk(), nv()>(pass, p, s); });
}
template <typename T>
hipError_t lin_fit_t(int64_t nk, int64_t nv, int *blocks) {
    return lin_sizes(nk, nv, [&](auto nk, auto nv) {
        static std::atomic<int> known{0};  // (a property of the compiled kernel)
        *blocks = known.load();
        if (*blocks > 0) return hipSuccess;
        hipError_t e;
        if constexpr (sizeof(T) == 2)
            e = hipOccupancyMaxActiveBlocksPerMultiprocessor(blocks, lin_output_kernel<nk(), nv()>, 2 * nv(), 0);
        else
            e = hipOccupancyMaxActiveBlocksPerMultiprocessor(
                blocks, lin_chunk_kernel<T, nk(), nv(), LinPass::kOutput>, 4 * nv(), 0);
        if (e == hipSuccess) known.store(*blocks);
        return e;
    });
}

// One decode step: h = L h + v k^T and y = scale h q.  A wave takes 8 rows of a
// state at a time (kRows of them, one behind the other), 8 lanes to a row; a
// lane holds four values of every 32.  Bound by the state's bytes.
constexpr int kLinStepRows = 2;
template <typename T, int kRuns>
__global__ __launch_bounds__(256) void lin_step_kernel(LinStepParams p, int64_t first) {
    const int lane = threadIdx.x % kWave, l8 = lane & 7;
    const int groups = (p.nv + 8 * kLinStepRows - 1) / (8 * kLinStepRows);
    const int64_t wave = first + (int64_t)blockIdx.x * 4 + uniform(threadIdx.x / kWave);
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
    const int64_t waves = p.Bsz * p.H * groups;
    constexpr int64_t kMost = int64_t(1) << 25;  // waves of a launch (its threads stay below 2^32)
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < waves && e == hipSuccess; first += kMost) {
        const int64_t n = waves - first < kMost ? waves - first : kMost;
        const dim3 grid((unsigned)((n + 3) / 4)), block(256);
        if (p.nk <= 32) hipLaunchKernelGGL((lin_step_kernel<T, 1>), grid, block, 0, s, p, first);
        else if (p.nk <= 64) hipLaunchKernelGGL((lin_step_kernel<T, 2>), grid, block, 0, s, p, first);
        else if (p.nk <= 96) hipLaunchKernelGGL((lin_step_kernel<T, 3>), grid, block, 0, s, p, first);
        else hipLaunchKernelGGL((lin_step_kernel<T, 4>), grid, block, 0, s, p, first);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace ssm
