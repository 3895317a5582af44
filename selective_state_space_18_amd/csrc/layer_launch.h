// Launchers of the gated recurrence and the layer norm (host side of
// gated_kernels.h and norm_kernels.h).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

// Gated linear recurrence (gated_kernels.h).  x, r, i, y [Bsz][L][Dm]; A [Dm];
// h_init, h_final [Bsz][Dm] ([nseq][Dm] for packed sequences, Bsz = 1); carry
// [Bsz][ceil(L / kGatedCarrySteps)][Dm]: the state before each tile's first
// step.  y, h_final and carry may be null (then not written).
constexpr int kGatedCarrySteps = 64;
constexpr int kGatedTileSteps = 128;  // most steps a block addresses with 32-bit offsets
// Sequence starts of 8 steps (bits), and the sequence that holds the step
// before them (-1: none).
struct GatedMark {
    int starts, before;
};
struct GatedParams {
    const void *x, *r, *i;
    const float *A, *h_init;
    void *y;
    float *h_final, *carry;
    int64_t Bsz, L, Dm;
    const int64_t *cu;  // packed sequences, or null
    int64_t nseq;
    int64_t carry_rows;  // ceil(L / kGatedCarrySteps)
    int cus;             // compute units of the device
    // set by the launchers (gated_kernels.h): sequence starts per 8 steps and the
    // chain of tiles
    GatedMark *marks;
    int links, groups, cols;  // tiles along time; channel groups of a row, of all rows
    float inv_groups, inv_cols;
    uint32_t *ticket, *states;
    uint64_t *pairs;
};
struct GatedBwdParams {
    GatedParams f;  // the forward's inputs; f.carry is read
    const void *dy;
    const float *dh_final;
    void *dx, *dr, *di;
    float *dA, *dh_init;
    float *part;  // set by the launchers: dA per tile and batch row
};
struct GatedStepParams {
    const void *x, *r, *i;
    const float *A, *h;
    float *h_out;
    void *y;
    int64_t Bsz, Dm;
};
// kPlan: *bytes of scratch and *blocks of the grid, nothing is launched;
// kPrepare: the scratch is initialised, and the outgoing states of empty
// sequences are written; kRun; kReduce (backward): dA.
enum class GatedPass { kPlan, kPrepare, kRun, kReduce };
struct GatedPlan {
    size_t bytes;
    int64_t blocks;
};
hipError_t gated_fwd_f32(GatedPass pass, GatedParams &p, void *scratch, GatedPlan *plan, hipStream_t s);
hipError_t gated_fwd_bf16(GatedPass pass, GatedParams &p, void *scratch, GatedPlan *plan, hipStream_t s);
hipError_t gated_bwd_f32(GatedPass pass, GatedBwdParams &q, void *scratch, GatedPlan *plan, hipStream_t s);
hipError_t gated_bwd_bf16(GatedPass pass, GatedBwdParams &q, void *scratch, GatedPlan *plan, hipStream_t s);
// to = from (or 0) for every row of states; with cu, of the empty sequences.
hipError_t gated_states(const int64_t *cu, int64_t rows, const float *from, float *to, int64_t Dm, hipStream_t s);
hipError_t gated_step_f32(const GatedStepParams &p, hipStream_t s);
hipError_t gated_step_bf16(const GatedStepParams &p, hipStream_t s);

// Layer norm (norm_kernels.h).  x, residual, sum, y, s, dy, dsum, dx
// [rows][Dm]; weight, bias, dweight, dbias [Dm]; mean, rstd [rows][Dm/group].
struct NormParams {
    const void *x, *residual;
    const float *weight, *bias;
    void *sum, *y;
    float *mean, *rstd;
    int64_t rows, Dm, group;
    float eps;
    int cus;  // compute units of the device
};
struct NormBwdParams {
    const void *s;
    const float *weight, *mean, *rstd;
    const void *dy, *dsum;
    void *dx;
    float *dweight, *dbias;
    int64_t rows, Dm, group;
    float *part;  // partial sums of dweight and dbias, or null (not wanted)
    int cus;
};
// kPlan: *bytes of scratch (part); kRun; kReduce: dweight, dbias from part.
enum class NormPass { kPlan, kRun, kReduce };
hipError_t norm_fwd_f32(const NormParams &p, hipStream_t s);
hipError_t norm_fwd_bf16(const NormParams &p, hipStream_t s);
hipError_t norm_bwd_f32(NormPass pass, NormBwdParams &p, size_t *bytes, hipStream_t s);
hipError_t norm_bwd_bf16(NormPass pass, NormBwdParams &p, size_t *bytes, hipStream_t s);

}  // namespace ssm
