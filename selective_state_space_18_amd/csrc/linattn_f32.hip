// Linear attention, fp32 storage, and the kernels that go by no storage type:
// the parts of packed sequences, states of empty ones, sums over a group's heads.
#include "linattn_kernels.h"

namespace ssm {

namespace {

// Steps of sequence k, wherever its borders lie.
__device__ __forceinline__ void lin_borders(const int64_t *cu, int64_t k, int64_t L, int64_t &begin, int64_t &end) {
    const int64_t a = cu[k], b = cu[k + 1];
    begin = a < 0 ? 0 : a > L ? L : a;
    end = b < begin ? begin : b > L ? L : b;
}

constexpr int kTableThreads = 1024, kTableBases = 4096;

// bases[k]: the parts of the sequences before k; slots[k]: those of them that are not
// a sequence's first.  Then every part looks its sequence up (the first bases are in
// LDS: a search takes a load per step).  One block: the sums run over all sequences.
// Valid sequences have L / seg_len parts with a predecessor at most; one that would
// pass that has no parts.
__global__ __launch_bounds__(kTableThreads) void lin_table_kernel(const int64_t *cu, int64_t nseq, int64_t L,
                                                                 int64_t seg_len, int64_t segs, int64_t *bases,
                                                                 int64_t *slots, LinSeg *table) {
    __shared__ int64_t sums[kTableThreads / kWave];
    __shared__ int some[kTableThreads / kWave];  // sequences with steps
    __shared__ int64_t near[kTableBases];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    int64_t before = 0, firsts = 0;
    for (int64_t k0 = 0; k0 < nseq; k0 += kTableThreads) {
        const int64_t k = k0 + tid;
        int64_t n = 0;
        if (k < nseq) {
            int64_t a, b;
            lin_borders(cu, k, L, a, b);
            n = (b - a + seg_len - 1) / seg_len;
        }
        int64_t up = n;  // sum up to this lane
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const int64_t v = __shfl_up(up, o);
            if (lane >= o) up += v;
        }
        const uint64_t with = __ballot(n > 0);
        if (lane == kWave - 1) sums[wave] = up, some[wave] = __popcll(with);
        __syncthreads();
        int64_t base = before, all = 0, first = firsts, every = 0;
        for (int w = 0; w < kTableThreads / kWave; ++w) {
            if (w < wave) base += sums[w], first += some[w];
            all += sums[w], every += some[w];
        }
        if (k < nseq) {
            bases[k] = base + up - n;
            slots[k] = base + up - n - first - __popcll(with & ((uint64_t(1) << lane) - 1));
            if (k < kTableBases) near[k] = base + up - n;
        }
        before += all;
        firsts += every;
        __syncthreads();
    }
    if (tid == 0) bases[nseq] = before;
    __threadfence_block();
    __syncthreads();
    const int64_t inner = nseq < kTableBases ? nseq : kTableBases;
    for (int64_t j = tid; j < segs; j += kTableThreads) {
        LinSeg s = {0, 0, 0, -1, 0};
        if (j < before) {
            int64_t lo = 0, hi = inner - 1;  // the last sequence with bases <= j
            if (inner < nseq && bases[inner] <= j) lo = inner, hi = nseq - 1;
            while (lo < hi) {
                const int64_t mid = (lo + hi + 1) / 2;
                if ((mid < kTableBases ? near[mid] : bases[mid]) <= j) lo = mid;
                else hi = mid - 1;
            }
            lin_borders(cu, lo, L, s.begin, s.end);
            const int64_t index = j - (lo < kTableBases ? near[lo] : bases[lo]), slot = slots[lo];
            if (slot + (s.end - s.begin - 1) / seg_len <= L / seg_len) {
                s.seq = (int32_t)lo;
                s.index = (int32_t)index;
                s.slot = (int32_t)(slot + index);
            }
        }
        table[j] = s;
    }
}

__global__ __launch_bounds__(256) void lin_states_kernel(const int64_t *cu, int64_t rows, int64_t L, const float *from,
                                                         float *to, int64_t count) {
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        if (cu) {
            int64_t a, b;
            lin_borders(cu, row, L, a, b);
            if (a < b) continue;
        }
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256)
            to[row * count + i] = from ? from[row * count + i] : 0.f;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void lin_group_sum_kernel(const float *src, T *dst, int64_t rows, int heads, int group,
                                                            int D, const int64_t *cu, int64_t nseq) {
    // packed: the sequences' steps alone (nothing was written to src for the others)
    int64_t from = 0, to = rows;
    if (cu) {
        const int64_t a = cu[0], b = cu[nseq];
        from = a < 0 ? 0 : a > rows ? rows : a;
        to = b < from ? from : b > rows ? rows : b;
    }
    from *= (int64_t)heads * D, to *= (int64_t)heads * D;
    // four values a thread; heads of a group are neighbours
    for (int64_t i = from + ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < to; i += (int64_t)gridDim.x * 1024) {
        const int64_t head = i / D;
        const float *a = src + head * group * D + (i - head * D);
        lin_f32x4 v = *reinterpret_cast<const lin_f32x4 *>(a);
        for (int j = 1; j < group; ++j) v += *reinterpret_cast<const lin_f32x4 *>(a + (int64_t)j * D);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[i + e] = from_acc<T>(v[e]);
    }
}

// The states that enter the parts of sequences of more than kLinDirect parts:
// states[i] = L^seg_len states[i-1] + (what part i-1 adds, in states[i]).  A
// thread takes four values of a head's state, kAhead parts in flight; blocks along y
// take sequences (a part that is not a sequence's last has seg_len steps).
__global__ __launch_bounds__(256) void lin_carry_kernel(LinParams p) {
    constexpr int kAhead = 8;
    const int64_t state = (int64_t)p.nk * p.nv;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= state * p.H) return;
    const int64_t pitch = state * p.H, rows = p.table ? p.nseq : p.Bsz;
    const int64_t *bases = p.bases;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        int64_t first, count;  // its parts' states
        if (p.table) {
            first = p.slots[row], count = bases[row + 1] - bases[row];
            if (first + count - 1 > p.L / p.seg_len) continue;
        } else {
            count = p.segs / p.Bsz, first = row * count;
        }
        const bool carries = count > kLinDirect;
        if (!carries && !p.copy_first) continue;
        const int h = (int)(at / state);
        const int e = (int)(at - h * state), col = e / p.nk, n = e % p.nk;
        float *s = p.states + first * pitch + at;
        double v[4] = {0.0, 0.0, 0.0, 0.0};
        if (p.h_init) {
            const float *from = p.h_init + (row * p.H + h) * state + (int64_t)col * p.sc + (int64_t)n * p.sn;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = (double)from[j * p.sn];
        }
        if (p.copy_first && count > 0)
            *reinterpret_cast<lin_f32x4 *>(s) = lin_f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
        if (!carries) continue;
        const double decay = exp((double)p.log_decay[h] * (double)p.seg_len);
        for (int64_t i = 1; i < count; i += kAhead) {
            lin_f32x4 add[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (i + j < count) add[j] = *reinterpret_cast<const lin_f32x4 *>(s + (i + j) * pitch);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (i + j >= count) break;
                lin_f32x4 sum;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    v[x] = fma_(decay, v[x], (double)add[j][x]);
                    sum[x] = (float)v[x];
                }
                *reinterpret_cast<lin_f32x4 *>(s + (i + j) * pitch) = sum;
            }
        }
    }
}

}  // namespace

hipError_t lin_table(const int64_t *cu, int64_t nseq, int64_t L, int64_t seg_len, int64_t segs, int64_t *bases,
                     int64_t *slots, LinSeg *table, hipStream_t s) {
    hipLaunchKernelGGL(lin_table_kernel, dim3(1), dim3(kTableThreads), 0, s, cu, nseq, L, seg_len, segs, bases, slots,
                       table);
    return hipGetLastError();
}

hipError_t lin_carry(const LinParams &p, hipStream_t s) {
    const int64_t rows = p.table ? p.nseq : p.Bsz, values = (int64_t)p.H * p.nk * p.nv;
    hipLaunchKernelGGL(lin_carry_kernel, dim3((unsigned)((values + 1023) / 1024), (unsigned)(rows < 256 ? rows : 256)),
                       dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t lin_states(const int64_t *cu, int64_t rows, int64_t L, const float *from, float *to, int64_t count,
                      hipStream_t s) {
    if (rows == 0 || count == 0 || to == nullptr) return hipSuccess;
    const int64_t x = (count + 1023) / 1024, y = rows < 4096 ? rows : 4096;
    hipLaunchKernelGGL(lin_states_kernel, dim3((unsigned)(x < 256 ? x : 256), (unsigned)y), dim3(256), 0, s, cu, rows, L,
                       from, to, count);
    return hipGetLastError();
}

hipError_t lin_group_sum(int dtype, const float *src, void *dst, int64_t rows, int heads, int group, int D,
                         const int64_t *cu, int64_t nseq, hipStream_t s) {
    const int64_t blocks = (rows * heads * D / 4 + 255) / 256;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (dtype == 0)
        hipLaunchKernelGGL(lin_group_sum_kernel<float>, grid, dim3(256), 0, s, src, static_cast<float *>(dst), rows,
                           heads, group, D, cu, nseq);
    else
        hipLaunchKernelGGL(lin_group_sum_kernel<bf16>, grid, dim3(256), 0, s, src, static_cast<bf16 *>(dst), rows,
                           heads, group, D, cu, nseq);
    return hipGetLastError();
}

int lin_chunk(int dtype) { return dtype == 0 ? lin_steps<float>() : lin_steps<bf16>(); }

hipError_t lin_fit_f32(int64_t nk, int64_t nv, int *blocks) { return lin_fit_t<float>(nk, nv, blocks); }
hipError_t lin_pass_f32(LinPass pass, const LinParams &p, hipStream_t s) { return lin_pass_t<float>(pass, p, s); }
hipError_t lin_step_f32(const LinStepParams &p, hipStream_t s) { return lin_step_t<float>(p, s); }

}  // namespace ssm
