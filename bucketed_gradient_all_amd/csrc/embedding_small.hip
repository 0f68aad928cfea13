// The embedding table's gradient for a small batch, in one launch.
//
// A workgroup owns a range of the table's rows and a slab of columns. It sorts
// the range's positions in LDS as the sorting kernel of the large path does
// (counts per wave, places, positions put in order), then its 16 waves sum the
// runs: each an equal part of the sorted positions, the runs that a part ends
// in joined through LDS. Every workgroup of a range sorts the same positions
// again; for a few thousand tokens that costs less than two more launches.
//
// What bounds it is latency (the chain token -> count -> place -> row of dout)
// or, if one token fills the batch, one compute unit's share of the memory
// bandwidth: the host's rule keeps that below 2 MB a workgroup. 2048 positions
// of 1024 fp32 columns, 30522 rows, a third of the positions padding: 8.4 us.
#include "embedding_kernels.h"

namespace ddp {
namespace {

constexpr int kGroups = kSmallTokens / kSortThreads;   // groups of 64 tokens a wave holds

template <class INDEX, int ACT, int GRAD, int VEC, bool ACC>
__global__ void __launch_bounds__(kSortThreads)
small_grad(EmbeddingArgs a, SmallPlan p, const INDEX *tokens, const void *dout, void *grad)
{
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t sums[kSortWaves];
    const int tid = int(threadIdx.x), lane = tid % 64, wave = wave_of();
    const int range_index = int(blockIdx.x) / p.slabs, slab = int(blockIdx.x) - range_index * p.slabs;
    const int lo = range_index * p.rows;
    const int rows = min(p.rows, int(a.n_rows) - lo);   // the range [lo, lo + rows)
    const int T = int(a.n_tokens);
    uint32_t *counts = lds;                             // [wave][row]
    uint32_t *begin = counts + kSortWaves * rows;       // [rows + 1]
    uint32_t *entry = begin + rows + 1;                 // [T] row in the range, position
    float *heads = reinterpret_cast<float *>(entry + T);   // [wave][VEC][64]
    for (int i = tid; i < rows * kSortWaves; i += kSortThreads) counts[i] = 0;
    __syncthreads();

    // count
    const Range range{uint64_t(a.first_row), uint64_t(lo), uint64_t(lo + rows)};
    const int part = (T + kSortThreads - 1) / kSortThreads * 64;
    const int from = min(T, part * wave), to = min(T, from + part);
    int held[kGroups];   // the row in the range, or -1
    if (from < to) {
        INDEX tok[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) tok[k] = ((const GLOBAL INDEX *)tokens)[min(from + k * 64 + lane, to - 1)];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const uint64_t r = range.row(tok[k]);
            const bool in = range.upto(r) && !range.below(r) && int64_t(r) != p.pad_row && from + k * 64 + lane < to;
            held[k] = in ? int(r) - lo : -1;
            if (in) atomicAdd(&counts[wave * rows + held[k]], 1u);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kGroups; ++k) held[k] = -1;
    }
    __syncthreads();

    // places: a thread has a row
    uint32_t n[kSortWaves], total = 0;
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) {
        n[k] = tid < rows ? counts[k * rows + tid] : 0;
        total += n[k];
    }
    uint32_t upto = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    uint32_t at = upto - total, all = 0;
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) {
        if (k < wave) at += sums[k];
        all += sums[k];
    }
    if (tid < rows) {
        begin[tid] = at;
#pragma unroll
        for (int k = 0; k < kSortWaves; ++k) {
            counts[k * rows + tid] = at;
            at += n[k];
        }
    }
    if (tid == 0) begin[rows] = all;
    __syncthreads();

    // put the positions in place: the lanes of a row find each other one row
    // after the other (few of 64 tokens are in the range)
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        uint64_t left = __ballot(held[k] >= 0);
        uint64_t same = 0;
        while (left) {
            const int row = __builtin_amdgcn_readlane(held[k], __ffsll((unsigned long long)left) - 1);
            const uint64_t peers = __ballot(held[k] == row);
            if (held[k] == row) same = peers;
            left &= ~peers;
        }
        if (held[k] >= 0) {
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            const int leader = __ffsll((unsigned long long)same) - 1;
            uint32_t place = 0;
            if (lane == leader) place = atomicAdd(&counts[wave * rows + held[k]], uint32_t(__popcll(same)));
            place = __shfl(place, leader) + rank;
            entry[place] = uint32_t(held[k]) << 16 | uint32_t(from + k * 64 + lane);
        }
    }
    __syncthreads();

    // sum: wave w has the entries [c0, c1)
    const Columns<VEC> c(slab, lane, a.width);
    const int entries = int(all), per = (entries + kSortWaves - 1) / kSortWaves;
    const int c0 = min(entries, per * wave), c1 = min(entries, c0 + per);
    float sum[VEC] = {};
    constexpr int AHEAD = 8;
    const auto keep_head = [&] {   // the sum of a run that an earlier wave began
#pragma unroll
        for (int j = 0; j < VEC; ++j) heads[(wave * VEC + j) * 64 + lane] = sum[j];
    };
    for (int base = c0; base < c1; base += 64) {
        const int i = base + lane, there = min(64, c1 - base);
        const uint32_t mine = entry[min(i, c1 - 1)];
        const int my_row = int(mine >> 16), my_pos = int(mine & 0xffff);
        const uint64_t last = __ballot(i < c1 && i == int(begin[my_row + 1]) - 1);
        const uint64_t head = __ballot(int(begin[my_row]) < c0);
        for (int e = 0; e < there; e += AHEAD) {
            typename Raw<ACT, VEC>::type x[AHEAD];
            typename Raw<GRAD, VEC>::type old[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int64_t pos = __builtin_amdgcn_readlane(my_pos, min(e + k, there - 1));
                x[k] = load<ACT, VEC>(dout, pos * a.act_stride + c.col);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (ACC && e + k < there && ((last & ~head) >> (e + k)) & 1) {
                    const int64_t row = lo + __builtin_amdgcn_readlane(my_row, e + k);
                    old[k] = load<GRAD, VEC>(grad, row * a.grad_stride + c.col);
                }
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {   // one wait for the batch, before its stores (see sum_runs)
                arrive(x[k]);
                if (ACC) arrive(old[k]);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (e + k < there) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) sum[j] = __fadd_rn(sum[j], widen<ACT>(x[k][j]));
                    if ((last >> (e + k)) & 1) {
                        if ((head >> (e + k)) & 1)
                            keep_head();
                        else
                            put<GRAD, VEC, ACC>(a, grad, lo + __builtin_amdgcn_readlane(my_row, e + k), c, old[k], sum);
#pragma unroll
                        for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
                    }
                }
            }
        }
    }
    // the run that goes on past this wave's part: its own if it begins here
    int tail_row = 0, tail_end = 0;
    bool open = false;
    if (c0 < c1) {
        tail_row = __builtin_amdgcn_readfirstlane(int(entry[c1 - 1] >> 16));
        tail_end = __builtin_amdgcn_readfirstlane(int(begin[tail_row + 1]));
        const int tail_begin = __builtin_amdgcn_readfirstlane(int(begin[tail_row]));
        open = tail_end > c1 && tail_begin >= c0;
        if (tail_end > c1 && tail_begin < c0) keep_head();
    }
    typename Raw<GRAD, VEC>::type old;
    if (ACC && open) old = load<GRAD, VEC>(grad, (lo + tail_row) * a.grad_stride + c.col);
    __syncthreads();
    if (open) {
        for (int w = wave + 1; w * per < tail_end; ++w) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] = __fadd_rn(sum[j], heads[(w * VEC + j) * 64 + lane]);
        }
        put<GRAD, VEC, ACC>(a, grad, lo + tail_row, c, old, sum);
    }
    if (!ACC && c.on) {
        const float none[VEC] = {};
        for (int r = wave; r < rows; r += kSortWaves)
            if (begin[r] == begin[r + 1]) store<GRAD, VEC>(grad, (lo + r) * a.grad_stride + c.col, none, c.skip);
    }
}

template <class INDEX, int ACT, int GRAD>
hipError_t small_types(const EmbeddingArgs &a, const SmallPlan &p, const INDEX *tokens, const void *dout, void *grad,
                       bool accumulate, hipStream_t s)
{
    constexpr int VEC = sum_vector(ACT, GRAD);
    const dim3 g(static_cast<unsigned>((a.n_rows + p.rows - 1) / p.rows * p.slabs)), b(kSortThreads);
    const unsigned lds = unsigned(sizeof(uint32_t) * (size_t(kSortWaves) * p.rows + p.rows + 1 + size_t(a.n_tokens) +
                                                      size_t(kSortWaves) * VEC * 64));
    if (accumulate)
        hipLaunchKernelGGL((small_grad<INDEX, ACT, GRAD, VEC, true>), g, b, lds, s, a, p, tokens, dout, grad);
    else
        hipLaunchKernelGGL((small_grad<INDEX, ACT, GRAD, VEC, false>), g, b, lds, s, a, p, tokens, dout, grad);
    return hipGetLastError();
}

template <class INDEX, int ACT>
hipError_t small_dtypes(const EmbeddingArgs &a, const SmallPlan &p, const INDEX *tokens, const void *dout, void *grad,
                        bool accumulate, hipStream_t s)
{
    switch (a.grad_dtype) {
    case DDP_F32: return small_types<INDEX, ACT, DDP_F32>(a, p, tokens, dout, grad, accumulate, s);
    case DDP_BF16: return small_types<INDEX, ACT, DDP_BF16>(a, p, tokens, dout, grad, accumulate, s);
    default: return small_types<INDEX, ACT, DDP_F16>(a, p, tokens, dout, grad, accumulate, s);
    }
}

template <class INDEX>
hipError_t small_index(const EmbeddingArgs &a, const SmallPlan &p, const INDEX *tokens, const void *dout, void *grad,
                       bool accumulate, hipStream_t s)
{
    switch (a.act_dtype) {
    case DDP_F32: return small_dtypes<INDEX, DDP_F32>(a, p, tokens, dout, grad, accumulate, s);
    case DDP_BF16: return small_dtypes<INDEX, DDP_BF16>(a, p, tokens, dout, grad, accumulate, s);
    default: return small_dtypes<INDEX, DDP_F16>(a, p, tokens, dout, grad, accumulate, s);
    }
}

}  // namespace

hipError_t launch_small_grad(const EmbeddingArgs &a, const SmallPlan &p, const void *tokens, const void *dout,
                             void *grad, bool accumulate, hipStream_t s)
{
    return a.index64 ? small_index(a, p, static_cast<const int64_t *>(tokens), dout, grad, accumulate, s)
                     : small_index(a, p, static_cast<const int32_t *>(tokens), dout, grad, accumulate, s);
}

}  // namespace ddp
