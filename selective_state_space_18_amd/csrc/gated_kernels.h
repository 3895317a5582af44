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
// Arithmetic is fp32 for both storage types, with exp2, sqrt, 1/x and 1/sqrt
// from the transcendental unit (each within about one ulp).  fp32 storage also
// carries the rounding of exp's argument, which bf16 storage does not need.
#pragma once

#include <type_traits>

#include "layer_launch.h"
#include "ssm_device.h"

namespace ssm {

// exp(v).  The product v log2(e) is rounded once; for fp32 storage what that
// and the constant's own rounding leave off (|v| up to 128; beyond, exp is 0 or
// inf) multiplies the result, so the relative error stays near one ulp instead
// of growing with |v|.
template <typename T>
__device__ __forceinline__ float exp_(float v) {
    const float t = v * kLog2e;
    if constexpr (sizeof(T) == 2) return fast_exp2(t);
    constexpr float kLow = 1.92596303e-8f, kLn2 = 0.69314718056f;  // log2(e) - kLog2e
    float off = __builtin_fmaf(v, kLow, __builtin_fmaf(v, kLog2e, -t));
    off = __builtin_fabsf(v) < 128.f ? off : 0.f;
    return fast_exp2(t) * __builtin_fmaf(off, kLn2, 1.f);
}

// 1 - a^2 is carried in units of 2^-24 and its root m in units of 2^-12: the root
// units read subnormal numbers as 0, and of a nearly closed gate 1 - a^2 is one
// (u = -1e-39) while its root is an ordinary number.  A root multiplies a gate,
// which is taken in units of 2^12 at no cost (gate_), so that a step has one
// product more: 1 to 2% of the forward's time (two more, 2 to 3%).
constexpr float kSquareUnits = 0x1p24f, kRootUnits = 0x1p12f;

// The logistic function.
template <typename T>
__device__ __forceinline__ float sigmoid_(float v) {
    return __builtin_amdgcn_rcpf(1.0f + exp_<T>(-v));
}
// The same in units of kRootUnits (below 2^-114 it is subnormal in them: 0).
template <typename T>
__device__ __forceinline__ float gate_(float v) {
    return __builtin_amdgcn_rcpf(__builtin_fmaf(exp_<T>(-v), kRootUnits, kRootUnits));
}

// Units of u = A s in which the exponent is taken: the kernels scale A by this
// once.  bf16 storage works in base-2 units.
template <typename T>
constexpr float kDecayUnits = sizeof(T) == 4 ? 1.0f : kLog2e;

// (1 - a^2) kSquareUnits for a = exp2(u2), u2 <= 0, and al = a kSquareUnits.  It
// cancels near 0; there it is 2 a sinh(v), v = -u2 ln2, with the series
// v (1 + v^2/6 + v^4/120 + v^6/5040) (the powers of ln2, the factor -2 and the
// units are in the coefficients), whose truncation for v < 0.5 is below
// v^8/362880 = 1.1e-8.
__device__ __forceinline__ float one_minus_square_(float u2, float a, float al) {
    constexpr float l = 0.69314718056f, l2 = l * l;
    constexpr float c0 = -2.0f * l * kSquareUnits, c1 = c0 * l2 / 6.0f, c2 = c0 * l2 * l2 / 120.0f,
                    c3 = c0 * l2 * l2 * l2 / 5040.0f;
    const float w = u2 * u2;
    const float near = (u2 * a) * __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(w, c3, c2), w, c1), w, c0);
    const float far = __builtin_fmaf(-al, a, kSquareUnits);
    return u2 > -0.5f * kLog2e ? near : far;
}

// The same from u <= 0 in kDecayUnits and a = exp(u).
template <typename T>
__device__ __forceinline__ float one_minus_square_of_(float u, float a, float al) {
    return one_minus_square_(sizeof(T) == 4 ? u * kLog2e : u, a, al);
}
// a = exp(u) and m = sqrt(1 - a^2) times kRootUnits.
template <typename T>
__device__ __forceinline__ void decay_(float u, float &a, float &m) {
    a = sizeof(T) == 4 ? exp_<T>(u) : fast_exp2(u);
    m = __builtin_amdgcn_sqrtf(one_minus_square_of_<T>(u, a, a * kSquareUnits));
}

// ---------------------------------------------------------------------------
// Work layout.
//
// A block of 8 waves holds one tile of the problem, kSteps consecutive steps
// of kCh channels of one batch row, entirely in registers: lane l of wave w
// has channels l V .. l V + V - 1 of the steps [w kRun, (w + 1) kRun).  Every
// input is read once and every output written once.
//
// A run of steps is the affine map h -> P h + H.  A tile reduces to one such
// pair per channel (waves through LDS), and tiles of one channel group are
// tied together through memory:
//   * each tile publishes its pair as one 64-bit word per channel;
//   * tiles form groups of kFan; the last tile of a group publishes the state
//     that leaves the group instead;
//   * a tile takes the state that left the previous group and folds the pairs
//     of the tiles before it in its own group, in order.
// The fold's order is fixed, so results do not depend on timing, and a value
// crosses the chip once per kFan tiles.  A word is its own flag: the scratch is
// filled with ones before the launch, all ones is "not there yet", and a pair
// or state that would be all ones (a NaN of that payload) is stored as another
// NaN.  Words are relaxed agent-scope atomics, so no other memory needs
// ordering by them.
//
// Waiting ends: blocks take their tiles from a counter, in the order of the
// chain.  A block only waits for tiles with lower numbers than its own, each
// taken by a block that is running and that works through its numbers in order;
// the lowest unfinished tile waits for nothing that has not been published.
//
// What bounds it: HBM.  Counters: every input is fetched once and every output
// written once; the chain adds 3% of writes to the forward of the 2.8B-shaped
// layer (4 x 16384 x 5120, bf16).  Its forward takes 0.49 ms (5.5 TB/s of its
// 8 bytes an element), the backward 0.98 ms (4.8 TB/s of 14 bytes).  2^20 x 1024:
// 1.66 ms (5.2 TB/s).  The vector units issue 0.14 and 0.17 instructions per SIMD
// and cycle, a third of their peak; a tile's arithmetic waits for its data, and its
// registers leave two blocks to a CU to cover that, so a product more in every step
// still shows (2% of the forward's time).  Short calls and rows of few columns are
// bound by the launches, by tiles too few for the chip and by the chain (2 to 2.5
// times the bytes' time for 1 x 2048 x 2560).
//
// Packed sequences: where a sequence starts, the map is constant (it takes
// nothing from before).  P = -0 marks such a map; products of decays are
// never -0 (exp >= +0).  A constant map is applied without its P, so a
// non-finite state of one sequence does not reach the next one.

constexpr int kGatedWaves = 8;
constexpr int kGatedFwdRun = 16;     // steps per wave, forward: 128-step tiles
constexpr int kGatedBwdRun = 8;      // backward: 64-step tiles
// Links per group of the chain, for kPer links to each wave; kPer = 0: every
// link passes its state on by itself.
template <int kPer>
constexpr int kGatedFan = kPer > 0 ? kPer * kGatedWaves : 1;
// Links whose words a wave reads at a time.
template <int kPer>
constexpr int kGatedTake = kPer > 1 ? 2 : 1;
constexpr int kGatedMarkSteps = 8;   // steps per entry of GatedParams::marks
static_assert(kGatedWaves * kGatedBwdRun == kGatedCarrySteps, "a backward tile starts from one row of the carry");
static_assert(kGatedWaves * kGatedFwdRun == 2 * kGatedCarrySteps, "a forward tile writes two rows of the carry");
static_assert(kGatedWaves * kGatedFwdRun == kGatedTileSteps, "the host's size limit");

template <int kPer>
constexpr bool kGatedLoop = kPer == 0;  // backward: blocks take several tiles

constexpr uint32_t kReset = 0x80000000u;  // bits of -0.0f
constexpr int32_t kBufOut = 0x7ffffff0;   // an offset past every buffer range

__device__ __forceinline__ bool is_reset(float P) { return __float_as_uint(P) == kReset; }

// (P, H) <- later after (P, H).
template <bool kPacked>
__device__ __forceinline__ void compose(float &P, float &H, float lP, float lH) {
    if (kPacked && is_reset(lP)) {
        P = lP;
        H = lH;
    } else {
        H = __builtin_fmaf(lP, H, lH);
        P = P * lP;
    }
}
template <bool kPacked>
__device__ __forceinline__ float apply(float P, float H, float in) {
    return kPacked && is_reset(P) ? H : __builtin_fmaf(P, in, H);
}

__device__ __forceinline__ uint64_t pair_word(float P, float H) {
    uint32_t p = __float_as_uint(P);
    if (p == 0xffffffffu) p = 0x7fc00000u;
    return (uint64_t)p | ((uint64_t)__float_as_uint(H) << 32);
}
__device__ __forceinline__ uint32_t state_word(float h) {
    const uint32_t u = __float_as_uint(h);
    return u == 0xffffffffu ? 0x7fc00000u : u;
}
template <typename W>
__device__ __forceinline__ W peek(const W *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W>
__device__ __forceinline__ void publish(W *p, W v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Where a block is: its tile along the chain, its batch row and channels.
struct GatedPlace {
    int link;     // position along the chain (backward: from the last tile)
    int64_t col;  // channel group, over all batch rows
    int64_t b;
    int c0;       // first channel of this lane
};

// q = n / d and the remainder, for 0 <= n < 2^23 and inv = 1.0f / d: the product
// is off by less than one, which the comparison puts right.  (The compiler's
// integer divisions, 64-bit ones above all, took 0.3 us at every block's start.)
__device__ __forceinline__ int quotient(int n, int d, float inv, int &rest) {
    int q = uniform((int)((float)n * inv));
    rest = n - q * d;
    if (rest < 0) {
        --q;
        rest += d;
    } else if (rest >= d) {
        ++q;
        rest -= d;
    }
    return q;
}

template <int V>
__device__ __forceinline__ GatedPlace gated_place(const GatedParams &p, int id) {
    GatedPlace w;
    int col, group;
    w.link = quotient(id, p.cols, p.inv_cols, col);
    w.col = col;
    w.b = quotient(col, p.groups, p.inv_groups, group);
    w.c0 = group * (kWave * V) + (threadIdx.x % kWave) * V;
    return w;
}
// The calling thread's next tile number (the counter starts at all ones, like
// the rest of the scratch).
__device__ __forceinline__ int gated_next(const GatedParams &p) {
    return (int)(atomicAdd(p.ticket, 1u) + 1u);
}
// The block's first tile (its only one where there is no chain).  What the
// tile's first loads need is read beside the counter, whose latency starts every
// block.
__device__ __forceinline__ int gated_first(const GatedParams &p, int *shared) {
    asm volatile("" ::"s"(p.x), "s"(p.r), "s"(p.i), "s"(p.L), "s"(p.Dm), "s"(p.cols), "s"(p.groups));
    int id = blockIdx.x;
    if (p.links > 1) {
        if (threadIdx.x == 0) *shared = gated_next(p);
        __syncthreads();
        id = uniform(*shared);
    }
    return id;
}

// Publishes what the links after this one wait for: the tile's pair (before
// its entering state is known), or from the last link of a group the state
// that leaves it.
template <int V, int kFan>
__device__ __forceinline__ void chain_pair(const GatedParams &p, const GatedPlace &w, const float (&P)[V],
                                           const float (&H)[V]) {
    if (w.link + 1 >= p.links || w.link % kFan == kFan - 1) return;
    uint64_t *dst = p.pairs + ((int64_t)w.link * p.cols + w.col) * (kWave * V) + (threadIdx.x % kWave) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) publish(dst + v, pair_word(P[v], H[v]));
}
template <int V, int kFan>
__device__ __forceinline__ void chain_state(const GatedParams &p, const GatedPlace &w, const float (&h)[V]) {
    if (w.link + 1 >= p.links || w.link % kFan != kFan - 1) return;
    uint32_t *dst =
        p.states + ((int64_t)(w.link / kFan) * p.cols + w.col) * (kWave * V) + (threadIdx.x % kWave) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) publish(dst + v, state_word(h[v]));
}

// What a wave reads of the chain at a time: the pairs of two links of the
// tile's group (wave z of the block has links z kPer .. of the group), and in
// the last wave, which has the fewest links before it, the state that left the
// group before.
template <int V, int kTake>
struct ChainWords {
    uint64_t pair[kTake][V];
    uint32_t state[V];
};

// Reads the words of the wave's first two links and the state, ready or not;
// chain_enter reads again those that were not there yet.
template <int V, int kPer>
__device__ __forceinline__ void chain_peek(const GatedParams &p, const GatedPlace &w, int wave,
                                           ChainWords<V, kGatedTake<kPer>> &c) {
    constexpr int kCh = kWave * V, kFan = kGatedFan<kPer>, kTake = kGatedTake<kPer>;
    const int pos = w.link % kFan, group = w.link / kFan;
    const int64_t stride = (int64_t)p.cols * kCh;
    const int64_t at = w.col * kCh + (threadIdx.x % kWave) * V;
    const uint64_t *src = p.pairs + (int64_t)(w.link - pos + wave * kPer) * stride + at;
#pragma unroll
    for (int k = 0; k < kTake; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) c.pair[k][v] = wave * kPer + k < pos ? peek(src + k * stride + v) : 0;
    if (wave == kGatedWaves - 1 && group > 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) c.state[v] = peek(p.states + (int64_t)(group - 1) * stride + at + v);
    }
}

// The state (or adjoint) that enters a tile: `first` for the first group of
// links, else through the published words.  Every wave calls it (it has a
// barrier) and gets the value of its lanes' channels.  sP, sH:
// [kGatedWaves][kCh].
template <bool kPacked, int V, int kPer>
__device__ __forceinline__ void chain_enter(const GatedParams &p, const GatedPlace &w, int wave,
                                            ChainWords<V, kGatedTake<kPer>> &c,
                                            const float (&first)[V], const float (&tP)[V], const float (&tH)[V],
                                            float (*sP)[kWave * V], float (*sH)[kWave * V], float *sIn,
                                            float (&in)[V]) {
    constexpr int kCh = kWave * V, kFan = kGatedFan<kPer>, kTake = kGatedTake<kPer>;
    const int lane = threadIdx.x % kWave;
    const int pos = w.link % kFan, group = w.link / kFan;
    const int64_t stride = (int64_t)p.cols * kCh;
    const int64_t at = w.col * kCh + lane * V;
    if (wave * kPer < pos) {
        const uint64_t *src = p.pairs + (int64_t)(w.link - pos + wave * kPer) * stride + at;
        const int n = pos - wave * kPer < kPer ? pos - wave * kPer : kPer;
        float P[V], H[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.f;
            H[v] = 0.f;
        }
#pragma unroll
        for (int k0 = 0; k0 < kPer; k0 += kTake) {
            if (k0 >= n) break;
            if (k0 > 0) {
#pragma unroll
                for (int k = 0; k < kTake; ++k)
#pragma unroll
                    for (int v = 0; v < V; ++v) c.pair[k][v] = k0 + k < n ? peek(src + (k0 + k) * stride + v) : 0;
            }
            for (;;) {
                bool wait = false;
#pragma unroll
                for (int k = 0; k < kTake; ++k)
#pragma unroll
                    for (int v = 0; v < V; ++v) wait |= c.pair[k][v] == ~(uint64_t)0;
                if (!wait) break;
                __builtin_amdgcn_s_sleep(1);
#pragma unroll
                for (int k = 0; k < kTake; ++k)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (k0 + k < n) c.pair[k][v] = peek(src + (k0 + k) * stride + v);
            }
#pragma unroll
            for (int k = 0; k < kTake; ++k)
                if (k0 + k < n)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        compose<kPacked>(P[v], H[v], __uint_as_float((uint32_t)c.pair[k][v]),
                                         __uint_as_float((uint32_t)(c.pair[k][v] >> 32)));
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sP[wave][lane * V + v] = P[v];
            sH[wave][lane * V + v] = H[v];
        }
    }
    if (wave == kGatedWaves - 1) {
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = first[v];
            if (group > 0) {
                const uint32_t *src = p.states + (int64_t)(group - 1) * stride + at + v;
                while (c.state[v] == 0xffffffffu) {
                    __builtin_amdgcn_s_sleep(1);
                    c.state[v] = peek(src);
                }
                h[v] = __uint_as_float(c.state[v]);
            }
            sIn[lane * V + v] = h[v];
        }
        if (kFan == 1) {  // the next link waits for this: at once
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = apply<kPacked>(tP[v], tH[v], h[v]);
            chain_state<V, kFan>(p, w, h);
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) in[v] = sIn[lane * V + v];
#pragma unroll
    for (int k = 0; k < kGatedWaves; ++k)
        if (k * kPer < pos)
#pragma unroll
            for (int v = 0; v < V; ++v) in[v] = apply<kPacked>(sP[k][lane * V + v], sH[k][lane * V + v], in[v]);
}

// A lane's channels of one step, as stored: a dword (two bf16 or one fp32), for
// kRowsLone a bf16.
// How the rows lie (kRows):
//   kRowsWhole: bf16 rows that are whole 64-byte pieces.  Their loads are
//     streamed (2% faster than through the caches).
//   kRowsPlain: dwords.  Loads keep the lines they touch in the caches, since
//     rows that are not whole lines share them with the next channel group (fp32,
//     777 channels: 69 us forward and 102 backward, against 85 and 134 when the
//     loads are streamed).
//   kRowsLoose: bf16 rows of an odd length, or tensors at odd multiples of two
//     bytes: the dwords straddle.  The last channel of an odd row is read with
//     the one before it and written by itself; `tail` is set in the blocks that
//     have it.  (Rows of one channel are read one by one.)
//   kRowsLone: such rows with one channel a lane, for the backward where fewer
//     than kGatedDenseCols columns share the chip.  Its stores are left to merge
//     in the cache.  (Forward / backward, loose against lone: 4 x 16384 x 5121
//     0.63 / 1.35 ms against 0.74 / 1.49, 3 x 5000 x 4001 141 / 283 us against
//     156 / 291, 20011 x 777 53 / 90 us against 54 / 81.)
enum : int { kRowsPlain = 0, kRowsWhole = 1, kRowsLoose = 2, kRowsLone = 3 };
// Channels of a lane.
template <typename T, int kRows>
constexpr int kGatedWidth = kRows == kRowsLone ? 1 : 4 / (int)sizeof(T);
struct GatedCols {
    int32_t from, to;  // offsets of the lane's dword in a row: loads, stores
    int32_t one;       // kRowsLoose: of its lone last channel
    int shift;
    bool tail;
};
template <typename T, int kRows>
__device__ __forceinline__ GatedCols gated_cols(const GatedParams &p, const GatedPlace &w) {
    constexpr int es = sizeof(T);
    const int32_t at = w.c0 * es;
    if constexpr (kRows == kRowsLoose) {
        const bool pair = w.c0 + 1 < p.Dm, lone = w.c0 + 1 == p.Dm;
        return {pair ? at : lone && p.Dm > 1 ? at - es : kBufOut, pair ? at : kBufOut, lone ? at : kBufOut,
                lone ? 8 * es : 0, p.Dm % 2 != 0 && uniform(w.c0) + kWave * 2 > p.Dm};
    }
    const int32_t in = w.c0 < p.Dm ? at : kBufOut;
    return {in, in, 0, 0, false};
}
template <int kRows>
__device__ __forceinline__ uint32_t load_step(__amdgpu_buffer_rsrc_t r, const GatedCols &c, int32_t soff) {
    if constexpr (kRows == kRowsLone)
        return (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, c.from, soff, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b32(r, c.from, soff, kRows == kRowsWhole ? kBufNt : 0);
}
// What the loads of a run of steps gave, for kRowsLoose.
template <int kRows, int kRun>
__device__ __forceinline__ void load_tail(const GatedParams &p, uint32_t (&u)[kRun], __amdgpu_buffer_rsrc_t r,
                                          const GatedCols &c, int j0, int32_t row_bytes) {
    if constexpr (kRows == kRowsLoose) {
        if (p.Dm == 1) {
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                u[j] = (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, c.one, (j0 + j) * row_bytes, 0);
        } else if (c.tail) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) u[j] >>= c.shift;
        }
    }
}
template <typename T>
__device__ __forceinline__ float unpack(uint32_t u, int v) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u);
    return __uint_as_float(v == 1 ? u & 0xffff0000u : u << 16);
}
template <typename T, int kRows, int V>
__device__ __forceinline__ void store_step(const float (&f)[V], __amdgpu_buffer_rsrc_t r, const GatedCols &c,
                                           int32_t soff) {
    static_assert(V == kGatedWidth<T, kRows>, "channels of a lane");
    uint32_t u;
    if constexpr (sizeof(T) == 4) {
        u = __float_as_uint(f[0]);
    } else if constexpr (kRows == kRowsLone) {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, from_acc<bf16>(f[0])), r, c.to, soff,
                                              0);
        return;
    } else {
        typedef bf16 pair_t __attribute__((ext_vector_type(2)));
        const pair_t q = {from_acc<bf16>(f[0]), from_acc<bf16>(f[1])};
        u = __builtin_bit_cast(uint32_t, q);
    }
    __builtin_amdgcn_raw_buffer_store_b32(u, r, c.to, soff, kRows == kRowsLoose ? 0 : kBufNt);
    if constexpr (kRows == kRowsLoose)
        if (c.tail) __builtin_amdgcn_raw_buffer_store_b16((unsigned short)u, r, c.one, soff, 0);
}

// The starts inside a wave's run of steps (bit j: step t + j starts a
// sequence), and the sequence that holds the step before the run (-1: none).
struct GatedStarts {
    uint32_t mask;
    int64_t k;
};
template <int kRun>
__device__ __forceinline__ GatedStarts gated_starts(const GatedParams &p, int64_t t, int valid) {
    GatedStarts r{0, -1};
    if (valid <= 0) return r;
    // scalar loads: the marks were written by an earlier kernel and do not
    // change while this one runs (they start at an even entry, and the array
    // has one entry more than its steps need)
    typedef const __attribute__((address_space(4))) int *Words;
    Words m = (Words)(uintptr_t)(p.marks + t / kGatedMarkSteps);
    r.k = m[1];
    r.mask = (uint32_t)m[0];
    if (kRun > kGatedMarkSteps && valid > kGatedMarkSteps) r.mask |= (uint32_t)m[2] << kGatedMarkSteps;
    r.mask &= (uint32_t)((1u << valid) - 1u);
    return r;
}
// The last sequence from k (which may be -1) on that starts at or before step t:
// steps that double, then halves.  Mostly it is the next one, but any number of
// sequences without steps may lie between (131072 of them behind the last step:
// 17 / 29 ms forward / backward one load after another, 0.05 / 0.05 so).
__device__ __forceinline__ int64_t seq_from(const int64_t *cu, int64_t nseq, int64_t k, int64_t t) {
    int64_t by = 1;
    while (k + by < nseq && cu[k + by] <= t) {
        k += by;
        by *= 2;
    }
    while ((by /= 2) > 0)
        if (k + by < nseq && cu[k + by] <= t) k += by;
    return k;
}
// The sequence that holds step t, for a sequence k at or before it.
__device__ __forceinline__ int64_t seq_forward(const GatedParams &p, int64_t k, int64_t t) {
    return seq_from(p.cu, p.nseq, k, t);
}
// The sequence that holds step t - 1, for the one that starts at t: the last one
// up to k that starts before t, or the first.
__device__ __forceinline__ int64_t seq_back(const GatedParams &p, int64_t k, int64_t t) {
    if (k <= 0 || p.cu[k] < t) return k;
    int64_t by = 1;
    while (k - by > 0 && p.cu[k - by] >= t) {
        k -= by;
        by *= 2;
    }
    // the result is in [k - by, k)
    int64_t lo = k > by ? k - by : 0;
    while (k - lo > 1) {
        const int64_t mid = (lo + k) / 2;
        if (p.cu[mid] < t)
            lo = mid;
        else
            k = mid;
    }
    return lo;
}
// Channel c of a row of states (null or no row: 0).
__device__ __forceinline__ float state_at(const float *s, int64_t row, int64_t Dm, int c) {
    return s != nullptr && row >= 0 && c < Dm ? s[row * Dm + c] : 0.f;
}

template <typename T, int V, bool kPacked, int kPer, int kRows>
__global__ __launch_bounds__(kGatedWaves * kWave) __attribute__((amdgpu_waves_per_eu(4))) void gated_fwd_kernel(
    GatedParams p) {
    constexpr int kRun = kGatedFwdRun, kSteps = kRun * kGatedWaves, kCh = kWave * V;
    constexpr int es = sizeof(T);
    __shared__ float sP[kGatedWaves][kCh], sH[kGatedWaves][kCh], cP[kGatedWaves][kCh], cH[kGatedWaves][kCh];
    __shared__ float sIn[kCh], sFirst[kCh];
    __shared__ int sId;
    const GatedPlace w = gated_place<V>(p, gated_first(p, &sId));
    // (after the place: 3% faster than before it)
    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const int64_t t0 = (int64_t)w.link * kSteps;
    const int rows = (int)(p.L - t0 < kSteps ? p.L - t0 : kSteps);
    const int row_bytes = (int)(p.Dm * es);
    const int64_t base = (w.b * p.L + t0) * row_bytes;
    const __amdgpu_buffer_rsrc_t bx = make_rsrc((const char *)p.x + base, rows * row_bytes);
    const __amdgpu_buffer_rsrc_t br = make_rsrc((const char *)p.r + base, rows * row_bytes);
    const __amdgpu_buffer_rsrc_t bi = make_rsrc((const char *)p.i + base, rows * row_bytes);
    const GatedCols cols = gated_cols<T, kRows>(p, w);
    const int j0 = wave * kRun;
    const int valid = rows - j0 < kRun ? rows - j0 : kRun;  // steps of this wave's run (may be <= 0)
    GatedStarts st{0, -1};
    if (kPacked) st = gated_starts<kRun>(p, t0 + j0, valid);
    uint32_t xr[kRun], rr[kRun], ir[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        rr[j] = load_step<kRows>(br, cols, (j0 + j) * row_bytes);
        ir[j] = load_step<kRows>(bi, cols, (j0 + j) * row_bytes);
        xr[j] = load_step<kRows>(bx, cols, (j0 + j) * row_bytes);
    }
    load_tail<kRows>(p, rr, br, cols, j0, row_bytes);
    load_tail<kRows>(p, ir, bi, cols, j0, row_bytes);
    load_tail<kRows>(p, xr, bx, cols, j0, row_bytes);
    float A[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = w.c0 + v < p.Dm ? p.A[w.c0 + v] * kDecayUnits<T> : 0.f;

    // every step's decay and input, then the run's maps from its start
    float P[kRun][V], H[kRun][V], cp[V], ch[V];
#pragma unroll
    for (int j = 0; j < kRun; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float m;
            decay_<T>(A[v] * sigmoid_<T>(unpack<T>(rr[j], v)), P[j][v], m);
            H[j][v] = m * gate_<T>(unpack<T>(ir[j], v)) * unpack<T>(xr[j], v);
        }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        cp[v] = 1.f;
        ch[v] = 0.f;
    }
    int64_t k = st.k;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        const bool start = kPacked && ((st.mask >> j) & 1u);
        if (start) {  // a first step takes its own initial state and nothing from before
            k = seq_forward(p, k, t0 + j0 + j);
#pragma unroll
            for (int v = 0; v < V; ++v) ch[v] = state_at(p.h_init, k, p.Dm, w.c0 + v);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            H[j][v] = ch[v] = __builtin_fmaf(P[j][v], ch[v], H[j][v]);
            P[j][v] = cp[v] = start ? -0.f : P[j][v] * cp[v];
        }
    }
    if (valid < kRun) {
        // steps past the row's end keep the state
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (j >= valid) {
                    P[j][v] = j > 0 ? P[j > 0 ? j - 1 : 0][v] : 1.f;
                    H[j][v] = j > 0 ? H[j > 0 ? j - 1 : 0][v] : 0.f;
                }
            cp[v] = P[kRun - 1][v];
            ch[v] = H[kRun - 1][v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sP[wave][lane * V + v] = cp[v];
        sH[wave][lane * V + v] = ch[v];
        // h_init is read here, before the barrier and so before this tile
        // publishes anything: h_final may be the same buffer, and the last
        // tile writes it once every tile before has published
        if (wave == kGatedWaves - 1)
            sFirst[lane * V + v] =
                kPacked || w.link >= kGatedFan<kPer> ? 0.f : state_at(p.h_init, w.b, p.Dm, w.c0 + v);
    }
    __syncthreads();
    // maps of the waves before this one, and of the whole tile
    float bP[V], bH[V], tP[V], tH[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bP[v] = tP[v] = 1.f;
        bH[v] = tH[v] = 0.f;
    }
#pragma unroll
    for (int q = 0; q < kGatedWaves; ++q)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (q == wave) {
                bP[v] = tP[v];
                bH[v] = tH[v];
            }
            compose<kPacked>(tP[v], tH[v], sP[q][lane * V + v], sH[q][lane * V + v]);
        }
    if (wave == 0) chain_pair<V, kGatedFan<kPer>>(p, w, tP, tH);

    float first[V], in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) first[v] = sFirst[lane * V + v];
    if (w.link == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) in[v] = first[v];
    } else {
        ChainWords<V, kGatedTake<kPer>> words;
        chain_peek<V, kPer>(p, w, wave, words);
        chain_enter<kPacked, V, kPer>(p, w, wave, words, first, tP, tH, cP, cH, sIn, in);
    }
    if (wave == 0) {
        float out[V];
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = apply<kPacked>(tP[v], tH[v], in[v]);
        if (kPer > 0 || w.link == 0) chain_state<V, kGatedFan<kPer>>(p, w, out);
    }
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = apply<kPacked>(bP[v], bH[v], in[v]);
    if (p.carry != nullptr && j0 % kGatedCarrySteps == 0 && valid > 0) {
        float *c = p.carry + (w.b * p.carry_rows + (t0 + j0) / kGatedCarrySteps) * p.Dm + w.c0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (w.c0 + v < p.Dm) c[v] = h[v];
    }
    const float enter[2] = {h[0], h[V - 1]};
    const __amdgpu_buffer_rsrc_t by = make_rsrc((char *)p.y + base, p.y != nullptr ? rows * row_bytes : 0);
    k = st.k;
    if (!kPacked || st.mask == 0) {
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(P[j][v], enter[v == 0 ? 0 : 1], H[j][v]);
            store_step<T, kRows>(h, by, cols, (j0 + j) * row_bytes);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            if ((st.mask >> j) & 1u) {
                // the state so far is the last one of the sequence before
                if (p.h_final != nullptr && k >= 0 && t0 + j0 + j > 0)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (w.c0 + v < p.Dm) p.h_final[k * p.Dm + w.c0 + v] = h[v];
                k = seq_forward(p, k, t0 + j0 + j);
            }
            const bool cut = (st.mask & ((2u << j) - 1u)) != 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = cut ? H[j][v] : __builtin_fmaf(P[j][v], enter[v == 0 ? 0 : 1], H[j][v]);
            store_step<T, kRows>(h, by, cols, (j0 + j) * row_bytes);
        }
    }
    if (t0 + rows == p.L && p.h_final != nullptr && valid > 0 && valid == rows - j0) {
        const int64_t row = kPacked ? k : w.b;  // (steps past the end kept the state)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (row >= 0 && w.c0 + v < p.Dm) p.h_final[row * p.Dm + w.c0 + v] = h[v];
    }
}

// Makes what is computed from v be computed here, not kept in registers from
// an earlier use of the same expression.
__device__ __forceinline__ void again_(float &v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void again_(uint32_t &v) { asm volatile("" : "+v"(v)); }

// m and a^2 / m (0 where m = 0), both times kRootUnits, from u and a.
template <typename T>
__device__ __forceinline__ void scale_again(float u, float a, float &m, float &quot) {
    again_(u);
    again_(a);
    const float al = a * kSquareUnits;
    const float m2 = one_minus_square_of_<T>(u, a, al);
    const float root = m2 > 0.f ? __builtin_amdgcn_rsqf(m2) : 0.f;
    m = m2 * root;
    quot = al * a * root;
}

template <typename T, int V, bool kPacked, int kPer, int kRows>
__global__ __launch_bounds__(kGatedWaves * kWave) __attribute__((amdgpu_waves_per_eu(4))) void gated_bwd_kernel(
    GatedBwdParams q) {
    // Where every link passes its state on, blocks stay and take tile after tile,
    // the next one's number fetched while this one's results are written: 7%
    // faster.  (The longer groups' kernels spill in such a loop, and the forward
    // is 10% slower with it.)
    constexpr bool kLoop = kGatedLoop<kPer>;
    constexpr int kRun = kGatedBwdRun, kSteps = kRun * kGatedWaves, kCh = kWave * V, kPeekAt = kRun / 2;
    constexpr int es = sizeof(T);
    const GatedParams &p = q.f;
    __shared__ float sP[kGatedWaves][kCh], sH[kGatedWaves][kCh], sE[kGatedWaves][kCh];
    __shared__ float cP[kGatedWaves][kCh], cH[kGatedWaves][kCh];
    __shared__ float sIn[kCh];
    __shared__ int sId;
    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const int tiles = p.links * p.cols;
    int id = gated_first(p, &sId), next = 0;
    // (a block that starts late, beside another stream's work, may find every
    // tile taken)
    while (!kLoop || id < tiles) {
        const GatedPlace w = gated_place<V>(p, id);
        const int tile = p.links - 1 - w.link;
        const int64_t t0 = (int64_t)tile * kSteps;
        const int rows = (int)(p.L - t0 < kSteps ? p.L - t0 : kSteps);
        int row_bytes = (int)(p.Dm * es);
        if (kLoop) asm volatile("" : "+s"(row_bytes));  // its multiples are not kept across tiles
        const int64_t base = (w.b * p.L + t0) * row_bytes;
        const __amdgpu_buffer_rsrc_t bx = make_rsrc((const char *)p.x + base, rows * row_bytes);
        const __amdgpu_buffer_rsrc_t br = make_rsrc((const char *)p.r + base, rows * row_bytes);
        const __amdgpu_buffer_rsrc_t bi = make_rsrc((const char *)p.i + base, rows * row_bytes);
        const __amdgpu_buffer_rsrc_t by = make_rsrc((const char *)q.dy + base, rows * row_bytes);
        const GatedCols cols = gated_cols<T, kRows>(p, w);
        const int j0 = wave * kRun;
        const int valid = rows - j0 < kRun ? rows - j0 : kRun;
        GatedStarts st{0, -1};
        if (kPacked) st = gated_starts<kRun>(p, t0 + j0, valid);
        uint32_t xr[kRun], rr[kRun], ir[kRun], yr[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            rr[j] = load_step<kRows>(br, cols, (j0 + j) * row_bytes);
            ir[j] = load_step<kRows>(bi, cols, (j0 + j) * row_bytes);
            xr[j] = load_step<kRows>(bx, cols, (j0 + j) * row_bytes);
            yr[j] = load_step<kRows>(by, cols, (j0 + j) * row_bytes);
        }
        load_tail<kRows>(p, rr, br, cols, j0, row_bytes);
        load_tail<kRows>(p, ir, bi, cols, j0, row_bytes);
        load_tail<kRows>(p, xr, bx, cols, j0, row_bytes);
        load_tail<kRows>(p, yr, by, cols, j0, row_bytes);
        float A[V], enter[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool on = w.c0 + v < p.Dm;
            A[v] = on ? p.A[w.c0 + v] * kDecayUnits<T> : 0.f;
            enter[v] = on ? p.carry[(w.b * p.carry_rows + tile) * p.Dm + w.c0 + v] : 0.f;
        }

        // Kept per step: the gates s and g, the decay a and the input b = m g x.  m is
        // computed again from a and u where the gradients use it: keeping their
        // coefficients instead (six values a step) needs more registers than four
        // waves per SIMD leave, and the spills cost more than everything else
        // (2.8B-shaped layer: 2.77 ms with them, 1.26 when they went, 0.98 now).
        float s[kRun][V], g[kRun][V], a[kRun][V], b[kRun][V];
        ChainWords<V, kGatedTake<kPer>> words;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            if (j == kPeekAt && w.link > 0) chain_peek<V, kPer>(p, w, wave, words);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[j][v] = sigmoid_<T>(unpack<T>(rr[j], v));
                g[j][v] = gate_<T>(unpack<T>(ir[j], v));
                float m;
                decay_<T>(A[v] * s[j][v], a[j][v], m);
                b[j][v] = m * g[j][v] * unpack<T>(xr[j], v);
            }
        }
        float pP[V], pH[V], pE[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            pP[v] = 1.f;
            pH[v] = 0.f;
            pE[v] = 0.f;
        }
        int64_t k = st.k;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const bool start = kPacked && ((st.mask >> j) & 1u);
            if (start) {
                k = seq_forward(p, k, t0 + j0 + j);
#pragma unroll
                for (int v = 0; v < V; ++v) pH[v] = state_at(p.h_init, k, p.Dm, w.c0 + v);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                pH[v] = __builtin_fmaf(a[j][v], pH[v], b[j][v]);
                pP[v] *= a[j][v];
            }
        }
        const int64_t k_end = k;  // the sequence of the run's last step
        if (valid < kRun) {
            // steps past the row's end (their inputs read as zeros) pass the
            // adjoint through and add nothing to dA: a = 1, s = 0
#pragma unroll
            for (int v = 0; v < V; ++v) {
                pP[v] = 1.f;
#pragma unroll
                for (int j = 0; j < kRun; ++j) {
                    if (j >= valid) {
                        a[j][v] = 1.f;
                        s[j][v] = 0.f;
                    }
                    pP[v] *= a[j][v];
                }
            }
        }
        // a start anywhere in the run makes its maps constant, whatever decays
        // (NaN among them) the steps around it have
        if (kPacked && st.mask != 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) pP[v] = -0.f;
        }
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) {
            const bool start = kPacked && ((st.mask >> j) & 1u);
            if (start) k = seq_back(p, k, t0 + j0 + j);
            again_(yr[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                pE[v] = a[j][v] * (unpack<T>(yr[j], v) + pE[v]);
                if (start) pE[v] = state_at(q.dh_final, k, p.Dm, w.c0 + v);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sP[wave][lane * V + v] = pP[v];
            sH[wave][lane * V + v] = pH[v];
            sE[wave][lane * V + v] = pE[v];
        }
        __syncthreads();
        // the adjoint maps of the waves after this one and of the whole tile, and
        // the state entering this wave's run
        float nP[V], nE[V], tP[V], tE[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nP[v] = tP[v] = 1.f;
            nE[v] = tE[v] = 0.f;
        }
#pragma unroll 2  // (eight at once hold 48 registers of loads)
        for (int z = kGatedWaves - 1; z >= 0; --z)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (z == wave) {
                    nP[v] = tP[v];
                    nE[v] = tE[v];
                }
                compose<kPacked>(tP[v], tE[v], sP[z][lane * V + v], sE[z][lane * V + v]);
            }
        if (wave == 0) chain_pair<V, kGatedFan<kPer>>(p, w, tP, tE);
#pragma unroll 2
        for (int z = 0; z < wave; ++z)
#pragma unroll
            for (int v = 0; v < V; ++v) enter[v] = apply<kPacked>(sP[z][lane * V + v], sH[z][lane * V + v], enter[v]);
        // (only the links of the first group use `first`)
        int64_t end = w.b;
        if (kPacked && w.link < kGatedFan<kPer>) end = seq_back(p, p.nseq - 1, p.L);
        float first[V], e[V];
#pragma unroll
        for (int v = 0; v < V; ++v) first[v] = e[v] = state_at(q.dh_final, end, p.Dm, w.c0 + v);
        if (w.link > 0) chain_enter<kPacked, V, kPer>(p, w, wave, words, first, tP, tE, cP, cH, sIn, e);
        if (wave == 0) {
            float out[V];
#pragma unroll
            for (int v = 0; v < V; ++v) out[v] = apply<kPacked>(tP[v], tE[v], e[v]);
            if (kPer > 0 || w.link == 0) chain_state<V, kGatedFan<kPer>>(p, w, out);
            if (!kPacked && tile == 0 && q.dh_init != nullptr)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (w.c0 + v < p.Dm) q.dh_init[w.b * p.Dm + w.c0 + v] = out[v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] = apply<kPacked>(nP[v], nE[v], e[v]);
        // the states before each step, in the place of b
        k = st.k;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            if (kPacked && ((st.mask >> j) & 1u)) {
                k = seq_forward(p, k, t0 + j0 + j);
#pragma unroll
                for (int v = 0; v < V; ++v) enter[v] = state_at(p.h_init, k, p.Dm, w.c0 + v);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float in = b[j][v];
                b[j][v] = enter[v];
                enter[v] = __builtin_fmaf(a[j][v], enter[v], in);
            }
        }

        if (kLoop && p.links > 1 && threadIdx.x == 0) next = gated_next(p);
        const __amdgpu_buffer_rsrc_t ox = make_rsrc((char *)q.dx + base, rows * row_bytes);
        const __amdgpu_buffer_rsrc_t orr = make_rsrc((char *)q.dr + base, rows * row_bytes);
        const __amdgpu_buffer_rsrc_t oi = make_rsrc((char *)q.di + base, rows * row_bytes);
        float dA[V];
#pragma unroll
        for (int v = 0; v < V; ++v) dA[v] = 0.f;
        k = k_end;
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) {
            float vx[V], vr[V], vi[V];
            again_(xr[j]);
            again_(yr[j]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float lam = unpack<T>(yr[j], v) + e[v], x = unpack<T>(xr[j], v), aj = a[j][v];
                float m, quot;
                scale_again<T>(A[v] * s[j][v], aj, m, quot);
                vx[v] = lam * (m * g[j][v]);
                vi[v] = vx[v] * x * __builtin_fmaf(g[j][v], -kRootUnits, 1.f);
                const float du = lam * (s[j][v] * (aj * b[j][v] - g[j][v] * x * quot));  // du s
                vr[v] = du * (A[v] * (1.f / kDecayUnits<T>) * (1.f - s[j][v]));
                dA[v] += du;
                e[v] = aj * lam;
            }
            store_step<T, kRows>(vx, ox, cols, (j0 + j) * row_bytes);
            store_step<T, kRows>(vr, orr, cols, (j0 + j) * row_bytes);
            store_step<T, kRows>(vi, oi, cols, (j0 + j) * row_bytes);
            if (j % 2 == 0) __builtin_amdgcn_sched_barrier(0);
            if (kPacked && ((st.mask >> j) & 1u)) {
                if (q.dh_init != nullptr && k >= 0)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (w.c0 + v < p.Dm) q.dh_init[k * p.Dm + w.c0 + v] = e[v];
                k = seq_back(p, k, t0 + j0 + j);
#pragma unroll
                for (int v = 0; v < V; ++v) e[v] = state_at(q.dh_final, k, p.Dm, w.c0 + v);
            }
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) sP[wave][lane * V + v] = dA[v];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float t = 0.f;
#pragma unroll
                for (int z = 0; z < kGatedWaves; ++z) t += sP[z][lane * V + v];
                if (w.c0 + v < p.Dm) q.part[((int64_t)tile * p.Bsz + w.b) * p.Dm + w.c0 + v] = t;
            }
        }
        if (!kLoop || p.links == 1) break;
        if (threadIdx.x == 0) sId = next;
        __syncthreads();
        id = uniform(sId);
    }
}

// What a scan needs before its tiles start, in one launch: the chain's words
// set to all ones; for packed sequences the marks, and the outgoing states of
// sequences without steps (to = from, or 0).  Without cu every row of states is
// copied.  (In launches of their own these cost about 3 us each.)
struct GatedPrepare {
    uint4 *words;
    int64_t nwords;
    const int64_t *cu;
    int64_t nseq, L, Dm;
    GatedMark *marks;
    int64_t nmarks;
    const float *from;
    float *to;
    int64_t mark_block, state_block, blocks;  // first blocks of the marks and the states; all blocks
};
__global__ __launch_bounds__(256) static void gated_prepare_kernel(GatedPrepare p) {
    if (blockIdx.x < p.mark_block) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (i < p.nwords) p.words[i] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
    } else if (blockIdx.x < p.state_block) {
        // sequence starts per kGatedMarkSteps steps
        const int64_t g = (blockIdx.x - p.mark_block) * 256 + threadIdx.x;
        if (g >= p.nmarks) return;
        const int64_t t = g * kGatedMarkSteps;
        // sequences that start before step t
        int64_t lo = 0, hi = p.nseq;
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (p.cu[mid] < t)
                lo = mid + 1;
            else
                hi = mid;
        }
        GatedMark m{0, (int)(lo - 1)};
        // (at most one start a step, from which the search goes on)
        for (int n = 0; n < kGatedMarkSteps && lo < p.nseq; ++n) {
            const int64_t d = p.cu[lo] - t;
            if (d >= kGatedMarkSteps) break;
            if (d >= 0) m.starts |= 1 << (int)d;
            lo = seq_from(p.cu, p.nseq, lo, p.cu[lo]) + 1;
        }
        p.marks[g] = m;
    } else {
        for (int64_t k = blockIdx.x - p.state_block; k < p.nseq; k += p.blocks - p.state_block) {
            if (p.cu != nullptr && p.cu[k] != p.cu[k + 1]) continue;
            for (int64_t c = threadIdx.x; c < p.Dm; c += 256)
                p.to[k * p.Dm + c] = p.from != nullptr ? p.from[k * p.Dm + c] : 0.f;
        }
    }
}

// dst[chunk][c] = sum of a chunk of `per` rows of src[rows][Dm]: 16 waves on
// every 16th row, eight rows in flight, then across the waves.  (21 MB of the
// 2.8B-shaped layer: 5.4 us, 3.9 TB/s.)
__global__ __launch_bounds__(1024) static void gated_sum_kernel(const float *__restrict__ src,
                                                                float *__restrict__ dst, int64_t rows, int64_t Dm,
                                                                int64_t per) {
    __shared__ float part[16][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWave + lane;
    const int64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
    float s = 0.f;
    if (c < Dm) {
        int64_t r = r0 + wave;
        for (; r + 7 * 16 < r1; r += 8 * 16) {
            float t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = src[(r + k * 16) * Dm + c];
#pragma unroll
            for (int k = 0; k < 8; ++k) s += t[k];
        }
        for (; r < r1; r += 16) s += src[r * Dm + c];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < Dm) {
        float t = 0.f;
#pragma unroll
        for (int z = 0; z < 16; ++z) t += part[z][lane];
        dst[blockIdx.y * Dm + c] = t;
    }
}

// One decode step.  A thread takes kVec consecutive channels of a row (16 bytes
// of state when kVec = 4), so a block reads A and walks rows without dividing.
// Bound by the launch: 256 x 8192 takes 6.5 us for 34 MB (5.2 TB/s, mostly from
// the caches), 4 x 1536 2.4 us; a call from Python takes 8 us of the host.
template <typename T, int kVec>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedStepParams p) {
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kVec;
    if (c >= p.Dm) return;
    struct alignas(kVec * sizeof(T)) In {
        T v[kVec];
    };
    struct alignas(kVec * 4) State {
        float v[kVec];
    };
    float A[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) A[k] = p.A[c + k] * kDecayUnits<T>;
    for (int64_t row = blockIdx.y; row < p.Bsz; row += gridDim.y) {
        const int64_t at = row * p.Dm + c;
        const In x = *reinterpret_cast<const In *>(static_cast<const T *>(p.x) + at);
        const In r = *reinterpret_cast<const In *>(static_cast<const T *>(p.r) + at);
        const In i = *reinterpret_cast<const In *>(static_cast<const T *>(p.i) + at);
        State h = *reinterpret_cast<const State *>(p.h + at);
        In y;
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            float a, m;
            decay_<T>(A[k] * sigmoid_<T>(to_f32(r.v[k])), a, m);
            h.v[k] = __builtin_fmaf(a, h.v[k], m * gate_<T>(to_f32(i.v[k])) * to_f32(x.v[k]));
            y.v[k] = from_acc<T>(h.v[k]);
        }
        *reinterpret_cast<State *>(p.h_out + at) = h;
        *reinterpret_cast<In *>(static_cast<T *>(p.y) + at) = y;
    }
}

// One pass's scratch in the layout of the kernels, the chain's words and then
// the marks; base may be null (sizes only).  per: links each wave folds.
// Returns the bytes; *chain: those of the words.
inline size_t gated_layout(GatedParams &p, int V, int steps, int per, char *base, size_t *chain) {
    const int64_t ch = kWave * V;
    p.groups = (int)((p.Dm + ch - 1) / ch);
    p.cols = (int)(p.Bsz * p.groups);  // (Bsz * Dm is below 2^30)
    p.inv_groups = 1.0f / (float)p.groups;
    p.inv_cols = 1.0f / (float)p.cols;
    p.links = (int)((p.L + steps - 1) / steps);
    const size_t all = (size_t)p.cols * ch;
    const int fan = per > 0 ? per * kGatedWaves : 1;
    const size_t states = p.links > 1 ? ((size_t)(p.links / fan) * all * 4 + 255) / 256 * 256 : 0;
    const size_t pairs = p.links > 1 && per > 0 ? (size_t)(p.links - 1) * all * 8 : 0;
    const size_t head = p.links > 1 ? 256 : 0;
    *chain = (head + states + pairs + 255) / 256 * 256;
    if (base != nullptr) {
        p.ticket = reinterpret_cast<uint32_t *>(base);
        p.states = reinterpret_cast<uint32_t *>(base + head);
        p.pairs = reinterpret_cast<uint64_t *>(base + head + states);
        p.marks = reinterpret_cast<GatedMark *>(base + *chain);
    }
    // (one entry more than the steps need: see gated_starts)
    const size_t marks = p.cu != nullptr ? (size_t)(p.L / kGatedMarkSteps + 2) * sizeof(GatedMark) : 0;
    return *chain + (marks + 255) / 256 * 256;
}

// Links each wave folds.  A group's state passes on in about 1.3 us, one group
// after another, while the columns (channel groups of all batch rows) share the
// chip's bandwidth; a tile takes about 0.025 us of that.  Longer groups hide the
// passing behind fewer columns, but a tile reads half a group's pairs.  Forward /
// backward times of bf16 layers:
//   kGatedDenseCols columns or more: 0.  Every link passes its state on: the
//     next tile of a column is further away than that, and no pairs are
//     written, cleared or read.  80 columns (4 x 16384 x 5120) 487 / 1043 us
//     against 507 / 1090 with groups of 16 links, and 980 with blocks that stay;
//     40 columns (65536 x 5120) 522 / 1124 against 504 / 1064 with groups of 8, 32
//     columns (65536 x 4096) 495 / 1075 against 398 / 844.
//   kGatedManyCols or more: 1 (8 links).  40 columns 504 / 1064 us against 507 /
//     1150 with 16 links, 16 columns (65536 x 2048) 220 / 446 against 224 / 476;
//     8 columns (131072 x 1024) 239 / 483 against 229 / 498.
//   one or two columns along many tiles: 8 (64 links); with 16 links the passing
//     alone is slower than the data (2^20 steps: 128 channels 0.69 / 1.31 ms with
//     16 links, 0.30 / 0.64 with 64; 512 channels 0.93 / 2.12 and 1.02 / 2.24).
//   else 2 (16 links); 4 columns (262144 x 512) 255 / 526 us against 358 / 680
//     with 8.
// The backward's columns of one channel (kRowsLone) carry half the bytes and so
// never pass link by link: 65536 x 5121, 81 of them, dense / packed, 1.49 / 1.55 ms
// with groups of 8 against 1.52 / 1.76, 65536 x 3201 1.03 / 1.00 against 1.10 / 1.19.
// From kGatedManyCols of them on 8 links are as good or better than 16: 65536 x 1025
// packed 348 us against 410.
constexpr int64_t kGatedDenseCols = 48, kGatedManyCols = 16, kGatedLongCols = 2, kGatedLongLinks = 256;
inline int gated_per(const GatedParams &p, int V, int steps) {
    const int64_t cols = p.Bsz * ((p.Dm + kWave * V - 1) / (kWave * V));
    if (cols >= kGatedDenseCols) return 0;
    if (cols >= kGatedManyCols) return 1;
    return cols <= kGatedLongCols && p.L / steps >= kGatedLongLinks ? 8 : 2;
}

// How the rows of a call's tensors lie (kRows above); dy, out[n]: a backward's.
template <typename T>
int gated_rows(const GatedParams &p, const void *dy, const void *const *out, int n) {
    if constexpr (sizeof(T) == 4) return kRowsPlain;
    const uintptr_t in = (uintptr_t)p.x | (uintptr_t)p.r | (uintptr_t)p.i | (uintptr_t)dy | (uintptr_t)(p.Dm * 2);
    uintptr_t all = in;
    for (int k = 0; k < n; ++k) all |= (uintptr_t)out[k];
    return all % 4 != 0 ? kRowsLoose : in % 64 == 0 ? kRowsWhole : kRowsPlain;
}

template <typename T, bool kPacked, int kPer, int kRows>
void gated_launch(const GatedParams &p, hipStream_t s) {
    hipLaunchKernelGGL((gated_fwd_kernel<T, kGatedWidth<T, kRows>, kPacked, kPer, kRows>),
                       dim3((unsigned)(p.links * p.cols)), dim3(kGatedWaves * kWave), 0, s, p);
}
template <typename T, bool kPacked, int kPer, int kRows>
void gated_launch(const GatedBwdParams &q, hipStream_t s) {
    // two blocks to a CU is what its registers hold
    const int64_t tiles = (int64_t)q.f.links * q.f.cols, held = 2 * (int64_t)q.f.cus;
    const int64_t blocks = kGatedLoop<kPer> && q.f.links > 1 && tiles > held ? held : tiles;
    hipLaunchKernelGGL((gated_bwd_kernel<T, kGatedWidth<T, kRows>, kPacked, kPer, kRows>), dim3((unsigned)blocks),
                       dim3(kGatedWaves * kWave), 0, s, q);
}
// p: the call's parameters (forward or backward).
template <typename T, bool kPacked, int kPer, typename Params>
void gated_pick(const Params &p, int rows, hipStream_t s) {
    constexpr bool kBwd = std::is_same<Params, GatedBwdParams>::value;
    if constexpr (sizeof(T) == 2) {
        if (rows == kRowsWhole) return gated_launch<T, kPacked, kPer, kRowsWhole>(p, s);
        if constexpr (!kBwd || kPer == 0)
            if (rows == kRowsLoose) return gated_launch<T, kPacked, kPer, kRowsLoose>(p, s);
        if constexpr (kBwd && kPer != 0)
            if (rows == kRowsLone) return gated_launch<T, kPacked, kPer, kRowsLone>(p, s);
    }
    gated_launch<T, kPacked, kPer, kRowsPlain>(p, s);
}
template <typename T, bool kPacked, typename Params>
void gated_pick(const Params &p, int per, int rows, hipStream_t s) {
    if (per == 0) gated_pick<T, kPacked, 0>(p, rows, s);
    else if (per == 1) gated_pick<T, kPacked, 1>(p, rows, s);
    else if (per == 2) gated_pick<T, kPacked, 2>(p, rows, s);
    else gated_pick<T, kPacked, 8>(p, rows, s);
}
template <typename T, typename Params>
void gated_pick(const Params &p, bool packed, int per, int rows, hipStream_t s) {
    if (packed) gated_pick<T, true>(p, per, rows, s);
    else gated_pick<T, false>(p, per, rows, s);
}

// to, from: outgoing and incoming states of the call, for sequences without
// steps (to may be null).
inline hipError_t gated_prepare(const GatedParams &p, size_t chain, const float *from, float *to, hipStream_t s) {
    GatedPrepare q{};
    q.words = reinterpret_cast<uint4 *>(p.ticket);
    q.nwords = (int64_t)(chain / 16);
    q.mark_block = q.state_block = q.blocks = (q.nwords + 255) / 256;
    q.cu = p.cu;
    q.nseq = p.nseq;
    q.L = p.L;
    q.Dm = p.Dm;
    q.from = from;
    q.to = to;
    if (p.cu != nullptr) {
        q.marks = p.marks;
        q.nmarks = (p.L + kGatedMarkSteps - 1) / kGatedMarkSteps;
        q.state_block = q.blocks = q.mark_block + (q.nmarks + 255) / 256;
        if (to != nullptr) q.blocks += p.nseq < 65536 ? p.nseq : 65536;
    }
    if (q.blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(gated_prepare_kernel, dim3((unsigned)q.blocks), dim3(256), 0, s, q);
    return hipGetLastError();
}
// to = from (or 0): every row of states, or with cu those of empty sequences.
inline hipError_t gated_states_launch(const int64_t *cu, int64_t rows, const float *from, float *to, int64_t Dm,
                                      hipStream_t s) {
    GatedPrepare q{};
    q.cu = cu;
    q.nseq = rows;
    q.Dm = Dm;
    q.from = from;
    q.to = to;
    q.blocks = rows < 65536 ? rows : 65536;
    if (rows == 0 || Dm == 0 || to == nullptr) return hipSuccess;
    hipLaunchKernelGGL(gated_prepare_kernel, dim3((unsigned)q.blocks), dim3(256), 0, s, q);
    return hipGetLastError();
}

template <typename T>
hipError_t gated_fwd_t(GatedPass pass, GatedParams &p, void *scratch, GatedPlan *plan, hipStream_t s) {
    const void *out[] = {p.y};
    const int V = 4 / (int)sizeof(T), rows = gated_rows<T>(p, nullptr, out, 1), per = gated_per(p, V, kGatedTileSteps);
    size_t chain;
    const size_t bytes = gated_layout(p, V, kGatedTileSteps, per, static_cast<char *>(scratch), &chain);
    if (pass == GatedPass::kPlan) {
        *plan = {bytes, (int64_t)p.links * p.cols};
        return hipSuccess;
    }
    if (pass == GatedPass::kPrepare) return gated_prepare(p, chain, p.h_init, p.h_final, s);
    gated_pick<T>(p, p.cu != nullptr, per, rows, s);
    return hipGetLastError();
}

// Rows each block of the dA sum adds, and the chunks of rows that makes.
constexpr int64_t kGatedSumRows = 1024;

template <typename T>
hipError_t gated_bwd_t(GatedPass pass, GatedBwdParams &q, void *scratch, GatedPlan *plan, hipStream_t s) {
    GatedParams &p = q.f;
    const void *out[] = {q.dx, q.dr, q.di};
    int form = gated_rows<T>(p, q.dy, out, 3), V = 4 / (int)sizeof(T);
    if (form == kRowsLoose && gated_per(p, V, kGatedCarrySteps) != 0) {
        form = kRowsLone;
        V = 1;
    }
    char *base = static_cast<char *>(scratch);
    int per = gated_per(p, V, kGatedCarrySteps);
    if (form == kRowsLone && per == 0) per = 1;
    size_t chain;
    const size_t head = gated_layout(p, V, kGatedCarrySteps, per, base, &chain);
    const int64_t rows = p.links * p.Bsz, chunks = (rows + kGatedSumRows - 1) / kGatedSumRows;
    const size_t part = ((size_t)(rows * p.Dm) * 4 + 255) / 256 * 256;
    const size_t sums = chunks > 1 ? ((size_t)(chunks * p.Dm) * 4 + 255) / 256 * 256 : 0;
    if (pass == GatedPass::kPlan) {
        *plan = {head + part + sums, (int64_t)p.links * p.cols};
        return hipSuccess;
    }
    q.part = reinterpret_cast<float *>(base + head);
    float *sum = reinterpret_cast<float *>(base + head + part);
    if (pass == GatedPass::kPrepare) return gated_prepare(p, chain, q.dh_final, q.dh_init, s);
    if (pass == GatedPass::kReduce) {
        const unsigned cols = (unsigned)((p.Dm + kWave - 1) / kWave);
        hipLaunchKernelGGL(gated_sum_kernel, dim3(cols, (unsigned)chunks), dim3(1024), 0, s, q.part,
                           chunks > 1 ? sum : q.dA, rows, p.Dm, kGatedSumRows);
        if (chunks > 1)
            hipLaunchKernelGGL(gated_sum_kernel, dim3(cols, 1), dim3(1024), 0, s, sum, q.dA, chunks, p.Dm, chunks);
        return hipGetLastError();
    }
    gated_pick<T>(q, p.cu != nullptr, per, form, s);
    return hipGetLastError();
}

template <typename T, int kVec>
void gated_step_run(const GatedStepParams &p, hipStream_t s) {
    const unsigned cols = (unsigned)((p.Dm + 256 * kVec - 1) / (256 * kVec));
    const unsigned rows = (unsigned)(p.Bsz < 65535 ? p.Bsz : 65535);
    hipLaunchKernelGGL((gated_step_kernel<T, kVec>), dim3(cols, rows), dim3(256), 0, s, p);
}

template <typename T>
hipError_t gated_step_t(const GatedStepParams &p, hipStream_t s) {
    // four channels a thread where rows and tensors allow 16-byte accesses to
    // the state (and 4 stored values at once); else one
    const uintptr_t in = (uintptr_t)p.x | (uintptr_t)p.r | (uintptr_t)p.i | (uintptr_t)p.y;
    const uintptr_t st = (uintptr_t)p.h | (uintptr_t)p.h_out;
    if (p.Dm % 4 == 0 && in % (4 * sizeof(T)) == 0 && st % 16 == 0)
        gated_step_run<T, 4>(p, s);
    else
        gated_step_run<T, 1>(p, s);
    return hipGetLastError();
}

}  // namespace ssm
