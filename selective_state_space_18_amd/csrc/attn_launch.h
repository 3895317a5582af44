// Launchers of linear attention (host side of linattn_kernels.h) and of the
// norm and rotation of queries and keys (qkrope_kernels.h).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

// One pass of linear attention over the sequences' steps, forwards or
// backwards in time.  The roles q, k, v of a pass are any of the call's tensors
// (the gradients are such passes, linattn_kernels.h); q and k have nk values a
// head, v and y nv.  A head h of the pass reads head h / gq of q, and so on.
constexpr int kLinMaxHead = 128;  // most values of a head
constexpr int64_t kLinMaxBlocks = int64_t(1) << 30;  // most parts of sequences times heads
// Up to so many parts of a sequence, the output pass sums what the parts before
// its own add by itself: n parts read (n - 1) / 2 states each, where carrying them
// first reads, writes and reads again.
constexpr int kLinDirect = 8;
// Part of a packed sequence: its steps `begin` .. `end` - 1, part number `index`
// of that sequence (-1: none), whose entry of the parts' states is `slot`.  A first part
// has no state of its own there: it shares the entry of the last part before it.
struct LinSeg {
    int64_t begin, end;
    int32_t seq, index, slot;
};
struct LinParams {
    const void *q, *k, *v;
    void *y;
    int y_f32;                 // y is fp32 whatever the storage type
    const float *log_decay;    // [H]
    const float *h_init;       // entering states, or null; element (col, n) of a
    float *h_final;            // state at col * sc + n * sn; h_final may be null
    int sc, sn;
    int64_t Bsz, L;
    int H, gq, gk, gv, nk, nv;
    int reverse;               // steps from the last to the first; a state that enters counts from its
                               // first step undecayed, one that leaves is decayed once more
    float y_scale, k_scale;    // y = y_scale * (...); sums of the states times k_scale
    int64_t seg_len;           // steps of a part (a multiple of lin_chunk())
    int64_t segs;              // parts of all sequences, at most
    const LinSeg *table;       // packed: the parts; null: segs / Bsz parts of every row
    const int64_t *bases;      // packed: the parts before each sequence's [nseq + 1]
    const int64_t *slots;      // packed: the entry of each sequence's first part [nseq]
    int64_t nseq;
    float *states;             // [segs][H] (packed: [L / seg_len + 1][H]) states that enter each part (of a
                               // sequence of up to kLinDirect parts: what the part before it adds); null: one
                               // part a row.  Element (col, n)
    int tc, tn;                // at col * tc + n * tn: nk and 1, but where another pass's states are read
    int copy_first;            // h_final may replace h_init: the first part's state is copied to `states`
    int first;                 // set by the launchers: the launch's first block of all of a pass
};
// The states that parts add; y.
enum class LinPass { kAggregate, kOutput };
int lin_chunk(int dtype);  // steps that a block takes at once
// Blocks of an output pass that a compute unit takes at once.
hipError_t lin_fit_f32(int64_t nk, int64_t nv, int *blocks);
hipError_t lin_fit_bf16(int64_t nk, int64_t nv, int *blocks);
hipError_t lin_pass_f32(LinPass pass, const LinParams &p, hipStream_t s);
hipError_t lin_pass_bf16(LinPass pass, const LinParams &p, hipStream_t s);
// The states that enter the parts, from what the aggregate pass left.
hipError_t lin_carry(const LinParams &p, hipStream_t s);
// The table of parts: bases is [nseq + 1] of scratch, slots [nseq].
hipError_t lin_table(const int64_t *cu, int64_t nseq, int64_t L, int64_t seg_len, int64_t segs, int64_t *bases,
                     int64_t *slots, LinSeg *table, hipStream_t s);
// to = from (or 0) for every row of `count` values; with cu, of sequences without steps.
hipError_t lin_states(const int64_t *cu, int64_t rows, int64_t L, const float *from, float *to, int64_t count,
                      hipStream_t s);
// dst[t][h][.] = sum of src[t][h * group + j][.] over j, rows of D values; with cu, of the steps from the
// first sequence's begin to the last one's end.
hipError_t lin_group_sum(int dtype, const float *src, void *dst, int64_t rows, int heads, int group, int D,
                         const int64_t *cu, int64_t nseq, hipStream_t s);
struct LinStepParams {
    const void *q, *k, *v;
    const float *log_decay, *h;
    float *h_out;
    void *y;
    int64_t Bsz;
    int H, group, nk, nv;
    float scale;
};
hipError_t lin_step_f32(const LinStepParams &p, hipStream_t s);
hipError_t lin_step_bf16(const LinStepParams &p, hipStream_t s);

// Norm and rotation of queries and keys (qkrope_kernels.h).  q, dq, q_out
// [rows][Hq][D]; k, dk, k_out [rows][Hk][D]; positions [rows]; freqs [R / 2];
// weights [D] or null.
constexpr int kRopeMaxHead = 1024;  // most values of a head
struct RopeParams {
    const void *q, *k, *dq, *dk;  // dq, dk: gradients of the outputs (backward)
    const int64_t *positions;
    const float *freqs, *q_weight, *k_weight;
    void *q_out, *k_out;          // the outputs, or (backward) the inputs' gradients
    float *dq_weight, *dk_weight;
    int64_t rows;
    int Hq, Hk, D, R, interleaved;
    float eps;
    float *part;                  // sums of dweight by blocks, or null (not wanted)
    int cus;                      // compute units of the device
    int tokens;                   // set by the launchers: tokens that a block takes at once
};
// kPlan: *bytes of scratch (part) of a backward; kReduce: dq_weight, dk_weight from part.
enum class RopePass { kForward, kPlan, kBackward, kReduce };
hipError_t rope_f32(RopePass pass, RopeParams &p, size_t *bytes, hipStream_t s);
hipError_t rope_bf16(RopePass pass, RopeParams &p, size_t *bytes, hipStream_t s);
hipError_t rope_reduce(const RopeParams &p, int64_t blocks, hipStream_t s);

}  // namespace ssm
