// Embedding lookup, and the table's gradient by sorted tokens.
//
//   out[t]  = R(scale * table[row(t)])
//   grad[v] = R([grad[v]] + scale * sum_{t: row(t) = v} dout[t])
//
// The lookup is a copy of rows: bound by memory, or by latency for few tokens.
//
// The gradient is a sum of rows of dout in an order that the tokens give. It
// runs in three launches without floating-point atomics, so that a call gives
// the same bits every time:
//   sort   each workgroup owns a range of the table's rows and looks through
//          all tokens, twice: it counts its rows' positions per wave (each wave
//          has a contiguous part of the tokens), turns the counts into places,
//          and puts its positions there in order. The workgroups share nothing:
//          where a range begins is the number of tokens of lower rows, which
//          each workgroup counts as it goes. Tokens are few bytes beside dout
//          and come from L2 after the first workgroup's read.
//   sum    a wave takes a chunk of the sorted positions and a slab of columns
//          and adds up run after run (the positions of one row). A run of at
//          most a chunk's length belongs to the chunk it begins in, which goes
//          beyond its end for it; only longer runs, of frequent tokens, are cut
//          at the chunks' borders into partial sums.
//   join   adds up the partial sums of the long runs.
#include "../../include/ddp.h"
#include "embedding.h"

#include <hip/hip_runtime.h>

namespace ddp {
namespace {

#define GLOBAL __attribute__((address_space(1)))

// VEC elements of a type as they lie in memory, at any element's address.
template <int TYPE, int VEC>
struct Raw;
template <int VEC>
struct Raw<DDP_F32, VEC> {
    typedef float type __attribute__((ext_vector_type(VEC)));
    typedef type any __attribute__((aligned(4)));
    typedef float elem;
};
template <int VEC>
struct Raw<DDP_BF16, VEC> {
    typedef unsigned short type __attribute__((ext_vector_type(VEC)));
    typedef type any __attribute__((aligned(2)));
    typedef unsigned short elem;
};
template <int VEC>
struct Raw<DDP_F16, VEC> : Raw<DDP_BF16, VEC> {};

template <int TYPE, class E>
__device__ __forceinline__ float widen(E v)
{
    if constexpr (TYPE == DDP_F32)
        return v;
    else if constexpr (TYPE == DDP_BF16)
        return __uint_as_float(uint32_t(v) << 16);
    else
        return float(__builtin_bit_cast(_Float16, v));
}

// One rounding to the type, to nearest even; beyond fp16's range it is inf.
template <int TYPE>
__device__ __forceinline__ typename Raw<TYPE, 1>::elem narrow(float v)
{
    if constexpr (TYPE == DDP_F32) {
        return v;
    } else if constexpr (TYPE == DDP_BF16) {
        return __builtin_bit_cast(unsigned short, static_cast<__bf16>(v));
    } else {
        asm volatile("" : "+v"(v));   // an fp32 value before the conversion (see `wire` in reduce_kernels.h)
        return __builtin_bit_cast(unsigned short, static_cast<_Float16>(v));
    }
}

template <int TYPE, int VEC>
__device__ __forceinline__ typename Raw<TYPE, VEC>::type load(const void *base, int64_t e)
{
    return *(const GLOBAL typename Raw<TYPE, VEC>::any *)(static_cast<const typename Raw<TYPE, VEC>::elem *>(base) + e);
}

// Columns of a lane: VEC of them from `col` on. The last lane of a row whose
// width is no multiple of VEC loads the row's last VEC columns instead, which
// overlap its neighbour's, and stores only its own: `skip` of them are the
// neighbour's. Rows narrower than VEC go one column a lane (VEC = 1).
template <int VEC>
struct Columns {
    int64_t col;
    int skip;
    bool on;
    __device__ __forceinline__ Columns(int64_t slab, int lane, int64_t width)
    {
        const int64_t c = (slab * 64 + lane) * VEC;
        on = c < width;
        col = c + VEC <= width ? c : width - VEC;
        skip = int(c - col);
        if (!on) col = 0, skip = 0;   // loads of an idle lane stay inside the row
    }
};

template <int TYPE, int VEC>
__device__ __forceinline__ void store(void *base, int64_t e, const float (&v)[VEC], int skip)
{
    typedef Raw<TYPE, VEC> R;
    typename R::elem *p = static_cast<typename R::elem *>(base) + e;
    if (skip == 0) {
        typename R::type x;
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = narrow<TYPE>(v[j]);
        *(GLOBAL typename R::any *)p = x;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (j >= skip) *(GLOBAL typename R::elem *)(p + j) = narrow<TYPE>(v[j]);
    }
}

// The row of the token at t, or -1.
__device__ __forceinline__ int row_of(const EmbeddingArgs &a, const void *tokens, int64_t t, bool drop_padding)
{
    const int64_t tok = a.index64 ? ((const GLOBAL int64_t *)tokens)[t] : int64_t(((const GLOBAL int32_t *)tokens)[t]);
    // unsigned, so that no index wraps into the range
    const uint64_t r = uint64_t(tok) - uint64_t(a.first_row);
    const bool pad = drop_padding && a.padding_idx >= 0 && tok == a.padding_idx;
    return r < uint64_t(a.n_rows) && !pad ? int(r) : -1;
}

constexpr int kWaves = 4;   // of a workgroup of the row kernels

__device__ __forceinline__ int wave_of()
{
    return __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 64);
}

// ---------------------------------------------------------------- lookup
// A wave copies a slab of 64 * VEC columns of TOK tokens' rows; all loads are
// issued before the first store.
template <int TABLE, int ACT, int VEC, int TOK>
__global__ void __launch_bounds__(kWaves * 64)
lookup(EmbeddingArgs a, int slabs, const void *table, const void *tokens, void *out)
{
    const int64_t task = int64_t(blockIdx.x) * kWaves + wave_of();
    const int64_t group = task / slabs;
    const int64_t t0 = group * TOK;
    if (t0 >= a.n_tokens) return;
    const Columns<VEC> c(task - group * slabs, int(threadIdx.x) % 64, a.width);
    int row[TOK];
    typename Raw<TABLE, VEC>::type x[TOK];
#pragma unroll
    for (int k = 0; k < TOK; ++k) row[k] = t0 + k < a.n_tokens ? row_of(a, tokens, t0 + k, false) : -1;
#pragma unroll
    for (int k = 0; k < TOK; ++k)
        if (row[k] >= 0) x[k] = load<TABLE, VEC>(table, row[k] * a.table_stride + c.col);
    if (!c.on) return;
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        if (t0 + k >= a.n_tokens) break;
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = row[k] >= 0 ? __fmul_rn(a.scale, widen<TABLE>(x[k][j])) : 0.0f;
        store<ACT, VEC>(out, (t0 + k) * a.act_stride + c.col, v, c.skip);
    }
}

// ---------------------------------------------------------------- sort
// Counters in LDS: counts[row in the range][wave], padded by a row's worth of
// nothing; a wave's 64 lanes hit different rows' counters.
__global__ void __launch_bounds__(kSortThreads) sort_tokens(EmbeddingArgs a, EmbeddingWork w, const void *tokens)
{
    extern __shared__ uint32_t counts[];   // [kSortWaves][rows]
    __shared__ uint32_t sums[kSortWaves];
    __shared__ uint32_t below_sums[kSortWaves];
    const int tid = int(threadIdx.x), lane = tid % 64, wave = wave_of();
    const int lo = int(blockIdx.x) * w.sort_rows;
    const int rows = min(w.sort_rows, int(a.n_rows) - lo);   // the range [lo, lo + rows)
    for (int i = tid; i < rows * kSortWaves; i += kSortThreads) counts[i] = 0;
    __syncthreads();

    // count
    const int T = int(a.n_tokens);
    const int part = (T + kSortThreads - 1) / kSortThreads * 64;
    const int from = int(min(int64_t(T), int64_t(part) * wave)), to = int(min(int64_t(T), int64_t(from) + part));
    uint32_t *mine = counts + wave * rows;
    uint32_t below = 0;
    constexpr int AHEAD = 8;
    for (int64_t i = from; i < to; i += 64 * AHEAD) {
        int r[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) r[k] = i + k * 64 + lane < to ? row_of(a, tokens, i + k * 64 + lane, true) : -1;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            below += r[k] >= 0 && r[k] < lo;
            if (r[k] >= lo && r[k] < lo + rows) atomicAdd(&mine[r[k] - lo], 1u);
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) below += __shfl_xor(below, d);
    if (lane == 0) below_sums[wave] = below;
    __syncthreads();

    // places: rows in order, a row's waves in order
    uint32_t base = 0;
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) base += below_sums[k];
    constexpr int PER = kMaxSortRows / kSortThreads;
    const int r0 = tid * PER;
    uint32_t n[PER], total = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        n[p] = 0;
        if (r0 + p < rows)
            for (int k = 0; k < kSortWaves; ++k) n[p] += counts[k * rows + r0 + p];
        total += n[p];
    }
    uint32_t upto = total;   // inclusive over the wave, then over the workgroup
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    uint32_t at = base + upto - total, all = base;
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) {
        if (k < wave) at += sums[k];
        all += sums[k];
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        if (r0 + p >= rows) break;
        w.begin[lo + r0 + p] = int(at);
        for (int k = 0; k < kSortWaves; ++k) {
            const uint32_t c = counts[k * rows + r0 + p];
            counts[k * rows + r0 + p] = at;
            at += c;
        }
    }
    if (tid == 0 && lo + rows == int(a.n_rows)) w.begin[a.n_rows] = int(all);
    __syncthreads();
    if (all == base) return;   // no position here

    // put the positions in place, each wave its own part in order: the lanes
    // of one row find each other by the bits of its number
    const int bits = 32 - __clz(max(rows - 1, 1));
    for (int64_t i = from; i < to; i += 64 * AHEAD) {
        int r[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) r[k] = i + k * 64 + lane < to ? row_of(a, tokens, i + k * 64 + lane, true) : -1;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const bool in = r[k] >= lo && r[k] < lo + rows;
            uint64_t same = __ballot(in);
            if (same == 0) continue;
            const int local = r[k] - lo;
            for (int b = 0; b < bits; ++b) {
                const uint64_t set = __ballot(in && ((local >> b) & 1));
                same &= (local >> b) & 1 ? set : ~set;
            }
            if (in) {
                const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
                const int leader = __ffsll((unsigned long long)same) - 1;
                uint32_t place = 0;
                if (lane == leader) place = atomicAdd(&mine[local], uint32_t(__popcll(same)));
                place = __shfl(place, leader) + rank;
                w.row[place] = r[k];
                w.pos[place] = int(i + k * 64 + lane);
            }
        }
    }
}

// ---------------------------------------------------------------- sum
template <int GRAD, int VEC>
__device__ __forceinline__ void put(const EmbeddingArgs &a, void *grad, bool accumulate, int row, const Columns<VEC> &c,
                                    const typename Raw<GRAD, VEC>::type &old, const float (&sum)[VEC])
{
    if (!c.on) return;
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        v[j] = accumulate ? __fmaf_rn(a.scale, sum[j], widen<GRAD>(old[j])) : __fmul_rn(a.scale, sum[j]);
    store<GRAD, VEC>(grad, row * a.grad_stride + c.col, v, c.skip);
}

template <int ACT, int GRAD, int VEC>
struct Summer {
    static constexpr int AHEAD = 8;   // rows of dout (and of grad, where a run ends) in flight
    const EmbeddingArgs &a;
    const EmbeddingWork &w;
    const Columns<VEC> &c;
    const void *dout;
    void *grad;
    bool accumulate;

    // the positions [i, end) of whole runs
    __device__ __forceinline__ void runs(int i, const int end) const
    {
        float sum[VEC] = {};
        while (i < end) {
            int row[AHEAD + 1];
            typename Raw<ACT, VEC>::type x[AHEAD];
            typename Raw<GRAD, VEC>::type old[AHEAD];
            bool last[AHEAD];
            const int n = min(AHEAD, end - i);
#pragma unroll
            for (int k = 0; k <= AHEAD; ++k) row[k] = w.row[min(i + k, end - 1)];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                last[k] = k < n && (i + k == end - 1 || row[k + 1] != row[k]);
                if (k < n) x[k] = load<ACT, VEC>(dout, w.pos[i + k] * a.act_stride + c.col);
                if (last[k] && accumulate) old[k] = load<GRAD, VEC>(grad, row[k] * a.grad_stride + c.col);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (k >= n) break;
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[j] = __fadd_rn(sum[j], widen<ACT>(x[k][j]));
                if (last[k]) {
                    put<GRAD, VEC>(a, grad, accumulate, row[k], c, old[k], sum);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
                }
            }
            i += n;
        }
    }

    // one piece of a long run
    __device__ __forceinline__ void piece(int i, const int end, float *slot) const
    {
        float sum[VEC] = {};
        while (i < end) {
            typename Raw<ACT, VEC>::type x[AHEAD];
            const int n = min(AHEAD, end - i);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (k < n) x[k] = load<ACT, VEC>(dout, w.pos[i + k] * a.act_stride + c.col);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (k >= n) break;
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum[j] = __fadd_rn(sum[j], widen<ACT>(x[k][j]));
            }
            i += n;
        }
        if (c.on) store<DDP_F32, VEC>(slot, c.col, sum, c.skip);
    }
};

template <int ACT, int GRAD, int VEC>
__global__ void __launch_bounds__(kWaves * 64)
sum_runs(EmbeddingArgs a, EmbeddingWork w, int slabs, int tasks, int accumulate, const void *dout, void *grad)
{
    const int task = int(blockIdx.x) * kWaves + wave_of();
    const int lane = int(threadIdx.x) % 64;
    if (task >= tasks) {
        // beyond the chunks: rows without a position, when the whole gradient
        // is written
        const int64_t z = int64_t(task) - (tasks + kWaves - 1) / kWaves * kWaves;
        const int64_t row = z / slabs;
        if (accumulate || z < 0 || row >= a.n_rows || w.begin[row] != w.begin[row + 1]) return;
        const Columns<VEC> c(z - row * slabs, lane, a.width);
        const float none[VEC] = {};
        if (c.on) store<GRAD, VEC>(grad, row * a.grad_stride + c.col, none, c.skip);
        return;
    }
    const int chunk = task / slabs;
    const Columns<VEC> c(task - chunk * slabs, lane, a.width);
    const int valid = w.begin[a.n_rows];
    const int i0 = chunk * w.chunk;
    if (i0 >= valid) return;
    const int border = min(i0 + w.chunk, valid);
    const Summer<ACT, GRAD, VEC> s{a, w, c, dout, grad, accumulate != 0};

    int i = i0, end = border;
    const int head = w.row[i0], head_begin = w.begin[head], head_end = w.begin[head + 1];
    if (head_begin < i0) {   // goes on from an earlier chunk: ours if it is long, that chunk's if not
        i = min(head_end, border);
        if (head_end - head_begin > w.chunk) s.piece(i0, i, w.more + int64_t(chunk) * w.pitch);
    }
    if (i >= border) return;
    const int tail = w.row[border - 1], tail_begin = w.begin[tail], tail_end = w.begin[tail + 1];
    if (tail_end > border) {   // goes on into the next chunk
        if (tail_end - tail_begin > w.chunk) {
            s.piece(tail_begin, border, w.first + int64_t(chunk) * w.pitch);
            end = tail_begin;
        } else {
            end = tail_end;
        }
    }
    s.runs(i, end);
}

// ---------------------------------------------------------------- join
constexpr int kJoinWaves = 16;

// The workgroup of the chunk in which a long run begins adds up the run's
// pieces: each wave a contiguous part of them, then the waves in order.
template <int GRAD, int VEC>
__global__ void __launch_bounds__(kJoinWaves * 64)
join_runs(EmbeddingArgs a, EmbeddingWork w, int slabs, int accumulate, void *grad)
{
    __shared__ float part[kJoinWaves][64 * VEC];
    const int chunk = int(blockIdx.x) / slabs, slab = int(blockIdx.x) - chunk * slabs;
    const int valid = w.begin[a.n_rows];
    const int i0 = chunk * w.chunk, border = i0 + w.chunk;
    if (border >= valid) return;
    const int row = w.row[border - 1], run_begin = w.begin[row], run_end = w.begin[row + 1];
    if (run_begin < i0 || run_end <= border || run_end - run_begin <= w.chunk) return;
    const int wave = wave_of(), lane = int(threadIdx.x) % 64;
    const Columns<VEC> c(slab, lane, a.width);
    const int pieces = (run_end - 1) / w.chunk - chunk;   // after the first
    const int each = (pieces + kJoinWaves - 1) / kJoinWaves;
    int k = chunk + 1 + wave * each;
    const int to = min(chunk + 1 + pieces, k + each);
    float sum[VEC] = {};
    constexpr int AHEAD = 8;
    while (k < to) {
        typename Raw<DDP_F32, VEC>::type x[AHEAD];
        const int n = min(AHEAD, to - k);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (j < n) x[j] = load<DDP_F32, VEC>(w.more + int64_t(k + j) * w.pitch, c.col);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (j >= n) break;
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum[e] = __fadd_rn(sum[e], x[j][e]);
        }
        k += n;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[wave][e * 64 + lane] = sum[e];
    __syncthreads();
    if (wave != 0) return;
    typename Raw<GRAD, VEC>::type old;
    if (accumulate) old = load<GRAD, VEC>(grad, row * a.grad_stride + c.col);
    const typename Raw<DDP_F32, VEC>::type x = load<DDP_F32, VEC>(w.first + int64_t(chunk) * w.pitch, c.col);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        sum[e] = x[e];
        for (int v = 0; v < kJoinWaves; ++v) sum[e] = __fadd_rn(sum[e], part[v][e * 64 + lane]);
    }
    put<GRAD, VEC>(a, grad, accumulate != 0, row, c, old, sum);
}

template <int VEC>
int slabs_of(int64_t width)
{
    return int((width + 64 * VEC - 1) / (64 * VEC));
}

template <int TABLE, int ACT, int VEC>
hipError_t lookup_vec(const EmbeddingArgs &a, const void *table, const void *tokens, void *out, hipStream_t s)
{
    const int64_t slabs = slabs_of<VEC>(a.width);
    // four rows a wave once that leaves every CU sixteen waves
    const bool four = a.n_tokens * slabs >= 4 * 256 * 16;
    const int64_t tasks = (four ? (a.n_tokens + 3) / 4 : a.n_tokens) * slabs;
    const dim3 g(unsigned((tasks + kWaves - 1) / kWaves)), b(kWaves * 64);
    if (four)
        hipLaunchKernelGGL((lookup<TABLE, ACT, VEC, 4>), g, b, 0, s, a, int(slabs), table, tokens, out);
    else
        hipLaunchKernelGGL((lookup<TABLE, ACT, VEC, 1>), g, b, 0, s, a, int(slabs), table, tokens, out);
    return hipGetLastError();
}

template <int TABLE, int ACT>
hipError_t lookup_types(const EmbeddingArgs &a, const void *table, const void *tokens, void *out, hipStream_t s)
{
    constexpr int VEC = TABLE == DDP_F32 ? 4 : 8;   // 16-byte loads
    return a.width >= VEC ? lookup_vec<TABLE, ACT, VEC>(a, table, tokens, out, s)
                          : lookup_vec<TABLE, ACT, 1>(a, table, tokens, out, s);
}

template <int TABLE>
hipError_t lookup_act(const EmbeddingArgs &a, const void *table, const void *tokens, void *out, hipStream_t s)
{
    switch (a.act_dtype) {
    case DDP_F32: return lookup_types<TABLE, DDP_F32>(a, table, tokens, out, s);
    case DDP_BF16: return lookup_types<TABLE, DDP_BF16>(a, table, tokens, out, s);
    default: return lookup_types<TABLE, DDP_F16>(a, table, tokens, out, s);
    }
}

template <int ACT, int GRAD, int VEC>
hipError_t sum_vec(const EmbeddingArgs &a, const void *dout, void *grad, bool accumulate, const EmbeddingWork &w,
                   hipStream_t s)
{
    const int64_t slabs = slabs_of<VEC>(a.width);
    const int64_t tasks = w.n_chunks * slabs;
    const int64_t fill = accumulate ? 0 : a.n_rows * slabs;
    const int64_t blocks = (tasks + kWaves - 1) / kWaves + (fill + kWaves - 1) / kWaves;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((sum_runs<ACT, GRAD, VEC>), dim3(unsigned(blocks)), dim3(kWaves * 64), 0, s, a, w, int(slabs),
                       int(tasks), accumulate ? 1 : 0, dout, grad);
    return hipGetLastError();
}

template <int ACT, int GRAD>
hipError_t sum_types(const EmbeddingArgs &a, const void *dout, void *grad, bool accumulate, const EmbeddingWork &w,
                     hipStream_t s)
{
    constexpr int VEC = ACT == DDP_F32 ? 4 : 8;
    return a.width >= VEC ? sum_vec<ACT, GRAD, VEC>(a, dout, grad, accumulate, w, s)
                          : sum_vec<ACT, GRAD, 1>(a, dout, grad, accumulate, w, s);
}

template <int ACT>
hipError_t sum_grad(const EmbeddingArgs &a, const void *dout, void *grad, bool accumulate, const EmbeddingWork &w,
                    hipStream_t s)
{
    switch (a.grad_dtype) {
    case DDP_F32: return sum_types<ACT, DDP_F32>(a, dout, grad, accumulate, w, s);
    case DDP_BF16: return sum_types<ACT, DDP_BF16>(a, dout, grad, accumulate, w, s);
    default: return sum_types<ACT, DDP_F16>(a, dout, grad, accumulate, w, s);
    }
}

template <int GRAD>
hipError_t join_grad(const EmbeddingArgs &a, void *grad, bool accumulate, const EmbeddingWork &w, hipStream_t s)
{
    const dim3 b(kJoinWaves * 64);
    if (a.width >= 4) {
        const int slabs = slabs_of<4>(a.width);
        hipLaunchKernelGGL((join_runs<GRAD, 4>), dim3(unsigned(int64_t(w.n_chunks) * slabs)), b, 0, s, a, w, slabs,
                           accumulate ? 1 : 0, grad);
    } else {
        hipLaunchKernelGGL((join_runs<GRAD, 1>), dim3(unsigned(w.n_chunks)), b, 0, s, a, w, 1, accumulate ? 1 : 0,
                           grad);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lookup(const EmbeddingArgs &a, const void *table, const void *tokens, void *out, hipStream_t s)
{
    switch (a.table_dtype) {
    case DDP_F32: return lookup_act<DDP_F32>(a, table, tokens, out, s);
    case DDP_BF16: return lookup_act<DDP_BF16>(a, table, tokens, out, s);
    default: return lookup_act<DDP_F16>(a, table, tokens, out, s);
    }
}

hipError_t launch_sort(const EmbeddingArgs &a, const void *tokens, const EmbeddingWork &w, hipStream_t s)
{
    const int groups = int((a.n_rows + w.sort_rows - 1) / w.sort_rows);
    const unsigned lds = unsigned(w.sort_rows) * kSortWaves * sizeof(uint32_t);
    hipLaunchKernelGGL(sort_tokens, dim3(unsigned(groups)), dim3(kSortThreads), lds, s, a, w, tokens);
    return hipGetLastError();
}

hipError_t launch_sum(const EmbeddingArgs &a, const void *dout, void *grad, bool accumulate, const EmbeddingWork &w,
                      hipStream_t s)
{
    switch (a.act_dtype) {
    case DDP_F32: return sum_grad<DDP_F32>(a, dout, grad, accumulate, w, s);
    case DDP_BF16: return sum_grad<DDP_BF16>(a, dout, grad, accumulate, w, s);
    default: return sum_grad<DDP_F16>(a, dout, grad, accumulate, w, s);
    }
}

hipError_t launch_join(const EmbeddingArgs &a, void *grad, bool accumulate, const EmbeddingWork &w, hipStream_t s)
{
    switch (a.grad_dtype) {
    case DDP_F32: return join_grad<DDP_F32>(a, grad, accumulate, w, s);
    case DDP_BF16: return join_grad<DDP_BF16>(a, grad, accumulate, w, s);
    default: return join_grad<DDP_F16>(a, grad, accumulate, w, s);
    }
}

}  // namespace ddp
