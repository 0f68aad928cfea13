// Embedding lookup, and the table's gradient by sorted tokens.
//
//   out[t]  = R(scale * table[row(t)])
//   grad[v] = R([grad[v]] + scale * sum_{t: row(t) = v} dout[t])
//
// The lookup is a copy of rows: bound by memory, or by latency for few tokens.
// 32767 rows of 2048 columns, half of them another shard's, fp32 into bf16: 23
// us, 172 MB.
//
// The gradient is a sum of rows of dout in an order that the tokens give. Small
// batches go another way (embedding_small.hip); here it runs in three launches
// without floating-point atomics, so that a call gives the same bits every time.
// 32768 positions of 2048 bf16 columns added to fp32, 32000 rows:
//   sort   14 us, bound by its instructions. Each workgroup looks after a range
//          of the table's rows. It looks through all tokens and counts its rows'
//          positions per part of the tokens, turns the counts into places, goes
//          through its parts again and puts its positions there in order. The
//          workgroups share nothing: where a range begins is the number of
//          tokens of lower rows, which each workgroup counts as it goes. Tokens
//          are few bytes beside dout and come from L2 after the first read.
//   sum    56 us, 290 MB at 5.2 TB/s, where plain streams reach 6.5; what holds
//          it below has not been told apart (lanes load 8 bytes of dout, and the
//          waves start behind three dependent loads). A wave takes a chunk of the
//          sorted positions and a slab of columns and adds up run after run (the
//          positions of one row). A run of at most a chunk's length belongs to
//          the chunk it begins in, which goes beyond its end for it; only longer
//          runs, of frequent tokens, are cut at the chunks' borders into partial
//          sums. Reading the gradient's old rows past the caches too took 63 us.
//   join   6 us, bound by latency: adds up the partial sums of the long runs.
#include "embedding_kernels.h"

namespace ddp {
namespace {

static_assert(kMaxSortRows <= 2 * kSortThreads);

// ---------------------------------------------------------------- lookup
// A wave copies a slab of 64 * VEC columns of TOK tokens' rows; all loads are
// issued before the first store.
// Workgroups of one wave: 32767 rows of 2048 columns 23.0 us against 24.4 with
// two waves and 26.1 with four; with two rows a wave 31.8, with eight 24.2.
constexpr int kLookupWaves = 1;
constexpr int kLookupRows = 4;

template <int TABLE, int ACT, int VEC, int TOK>
__global__ void __launch_bounds__(kLookupWaves * 64)
lookup(EmbeddingArgs a, int slabs, const void *table, const void *tokens, void *out)
{
    const int task = int(blockIdx.x) * kLookupWaves + wave_of();
    const int group = task / slabs;
    const int64_t t0 = int64_t(group) * TOK;
    if (t0 >= a.n_tokens) return;
    const Columns<VEC> c(task - group * slabs, int(threadIdx.x) % 64, a.width);
    int row[TOK];
    typename Raw<TABLE, VEC>::type x[TOK];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const int64_t t = min(t0 + k, a.n_tokens - 1);   // past the end: the last one again
        row[k] = row_of(a, a.index64 ? ((const CONSTANT int64_t *)tokens)[t] : ((const CONSTANT int32_t *)tokens)[t]);
    }
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
// Calls f(row, in range?, position) for the tokens [from, to) in order, 64 at
// a time, and adds up those below the range. The loads of eight groups are in
// flight together.
constexpr int kSortAhead = 8;

template <class INDEX, class F>
__device__ __forceinline__ uint32_t each_token(const Range &range, const INDEX *tokens, int from, int to, int lane, F f)
{
    constexpr int AHEAD = kSortAhead;
    const GLOBAL INDEX *p = (const GLOBAL INDEX *)tokens;
    uint32_t below = 0;
    int i = from;
    for (; i + 64 * AHEAD <= to; i += 64 * AHEAD) {
        INDEX tok[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) tok[k] = p[i + k * 64 + lane];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const uint64_t r = range.row(tok[k]);
            const bool low = range.below(r);
            below += __popcll(__ballot(low));
            f(r, range.upto(r) && !low, i + k * 64 + lane);
        }
    }
    if (i < to) {   // the rest, with the last token in the place of those past it
        INDEX tok[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) tok[k] = p[min(i + k * 64 + lane, to - 1)];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const bool there = i + k * 64 + lane < to;
            const uint64_t r = range.row(tok[k]);
            const bool low = range.below(r);
            below += __popcll(__ballot(low && there));
            f(r, range.upto(r) && !low && there, i + k * 64 + lane);
        }
    }
    return below;
}

// The tokens are cut into 16 * splits parts. The workgroups of one range are
// `splits` many: each counts all parts and puts 16 of them in place, one a
// wave. Putting in place costs most for the range of a frequent token (most
// groups of 64 tokens hold one), and that is the time of the whole kernel.
//
// Counters in LDS: [part of this workgroup][row], then the rows' sums over the
// parts of earlier and of later workgroups.
// HELD: a wave's part is at most eight groups of 64 tokens, which stay in its
// registers from the count on.
template <class INDEX, int PER, bool HELD>
__global__ void __launch_bounds__(kSortThreads) sort_tokens(EmbeddingArgs a, EmbeddingWork w, const INDEX *tokens)
{
    extern __shared__ uint32_t counts[];
    __shared__ uint32_t sums[kSortWaves];
    __shared__ uint32_t below_sums[kSortWaves];
    const int tid = int(threadIdx.x), lane = tid % 64, wave = wave_of();
    const int split = int(blockIdx.x) % w.splits;
    const int lo = int(blockIdx.x) / w.splits * w.sort_rows;
    const int rows = min(w.sort_rows, int(a.n_rows) - lo);   // the range [lo, lo + rows)
    const Range range{uint64_t(a.first_row), uint64_t(lo), uint64_t(lo + rows)};
    for (int i = tid; i < rows * (kSortWaves + 2); i += kSortThreads) counts[i] = 0;
    __syncthreads();

    // count
    const int64_t T = a.n_tokens;
    const int parts = kSortWaves * w.splits;
    const int64_t part = (T + parts * 64 - 1) / (parts * 64) * 64;
    uint32_t *mine = counts + wave * rows;
    uint32_t *earlier = counts + kSortWaves * rows, *later = earlier + rows;
    uint32_t below = 0;
    int my_from = 0, my_to = 0;
    int held[kSortAhead];   // the row in the range, or -1
    for (int q = 0; q < w.splits; ++q) {
        const int from = int(min(T, part * (q * kSortWaves + wave))), to = int(min(T, from + part));
        if (q == split) my_from = from, my_to = to;
        uint32_t *to_here = q == split ? mine : (q < split ? earlier : later);
        if constexpr (HELD) {
            INDEX tok[kSortAhead];
#pragma unroll
            for (int k = 0; k < kSortAhead; ++k)   // past the part: its last token, or for an empty part the first
                tok[k] = ((const GLOBAL INDEX *)tokens)[max(0, min(from + k * 64 + lane, to - 1))];
#pragma unroll
            for (int k = 0; k < kSortAhead; ++k) {
                const bool there = from + k * 64 + lane < to;
                const uint64_t r = range.row(tok[k]);
                const bool low = range.below(r);
                below += __popcll(__ballot(low && there));
                const bool in = range.upto(r) && !low && there;
                held[k] = in ? int(r) - lo : -1;
                if (in) atomicAdd(&to_here[held[k]], 1u);
            }
        } else {
            below += each_token(range, tokens, from, to, lane, [&](uint64_t r, bool in, int) {
                if (in) atomicAdd(&to_here[int(r) - lo], 1u);
            });
        }
    }
    if (lane == 0) below_sums[wave] = below;
    __syncthreads();

    // places: rows in order, a row's parts in order
    uint32_t base = 0;
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) base += below_sums[k];
    uint32_t n[PER][kSortWaves], before[PER], total[PER], mine_total = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int r = tid * PER + p;
        const bool there = r < rows;
        before[p] = there ? earlier[r] : 0;
        total[p] = before[p] + (there ? later[r] : 0);
#pragma unroll
        for (int k = 0; k < kSortWaves; ++k) {
            n[p][k] = there ? counts[k * rows + r] : 0;
            total[p] += n[p][k];
        }
        mine_total += total[p];
    }
    uint32_t upto = mine_total;   // inclusive over the wave, then over the workgroup
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    uint32_t at = base + upto - mine_total, all = base;
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) {
        if (k < wave) at += sums[k];
        all += sums[k];
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int r = tid * PER + p;
        if (r < rows) {
            if (split == 0) w.begin[lo + r] = int(at);
            uint32_t here = at + before[p];
#pragma unroll
            for (int k = 0; k < kSortWaves; ++k) {
                counts[k * rows + r] = here;
                here += n[p][k];
            }
        }
        at += total[p];
    }
    if (split == 0 && tid == 0 && lo + rows == int(a.n_rows)) w.begin[a.n_rows] = int(all);
    __syncthreads();
    if (all == base) return;   // no position here

    // Put the positions in place, each wave its own part in order. The lanes of
    // one row have to find each other. Mostly there are few rows among 64
    // tokens (none, or a frequent one): they are taken one by one. Where more
    // than kPeel are left, all find each other by the bits of their numbers,
    // which costs the same however many there are.
    constexpr int kPeel = 4;
    const int bits = 32 - __clz(max(rows - 1, 1));
    const auto place_group = [&](int local, bool in, int pos) {
        uint64_t left = __ballot(in);
        if (left == 0) return;
        uint64_t same = 0;   // the lanes of this lane's row
        for (int k = 0; left && k < kPeel; ++k) {
            const int row = __builtin_amdgcn_readlane(local, __ffsll((unsigned long long)left) - 1);
            const uint64_t peers = __ballot(in && local == row);
            if (local == row) same = peers;
            left &= ~peers;
        }
        if (left) {
            uint64_t mine_too = left;
            for (int b = 0; b < bits; ++b) {
                const bool bit = (local >> b) & 1;
                const uint64_t set = __ballot(bit);
                mine_too &= bit ? set : ~set;
            }
            if ((left >> lane) & 1) same = mine_too;
        }
        if (in) {
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            const int leader = __ffsll((unsigned long long)same) - 1;
            uint32_t place = 0;
            if (lane == leader) place = atomicAdd(&mine[local], uint32_t(__popcll(same)));
            place = __shfl(place, leader) + rank;
            w.row[place] = lo + local;
            w.pos[place] = pos;
        }
    };
    if constexpr (HELD) {
#pragma unroll
        for (int k = 0; k < kSortAhead; ++k) place_group(held[k], held[k] >= 0, my_from + k * 64 + lane);
    } else {
        each_token(range, tokens, my_from, my_to, lane,
                   [&](uint64_t r, bool in, int pos) { place_group(int(r) - lo, in, pos); });
    }
}

// ---------------------------------------------------------------- sum
// Task z of writing zeros over a slab of a row without a position, from row
// `from` on, when the whole gradient is written.
template <int GRAD, int VEC>
__device__ __forceinline__ void fill_row(const EmbeddingArgs &a, const EmbeddingWork &w, int slabs, int z, int64_t from,
                                         void *grad)
{
    const CONSTANT int32_t *begin = (const CONSTANT int32_t *)w.begin;
    const int64_t row = from + z / slabs;
    if (row >= a.n_rows || (begin[row] != begin[row + 1] && row != w.pad_row)) return;
    const Columns<VEC> c(z % slabs, int(threadIdx.x) % 64, a.width);
    const float none[VEC] = {};
    if (c.on) store<GRAD, VEC>(grad, row * a.grad_stride + c.col, none, c.skip);
}

template <int GRAD, int VEC>
__global__ void __launch_bounds__(kWaves * 64)
fill_rows(EmbeddingArgs a, EmbeddingWork w, int slabs, int tasks, int64_t from, void *grad)
{
    const int z = int(blockIdx.x) * kWaves + wave_of();
    if (z < tasks) fill_row<GRAD, VEC>(a, w, slabs, z, from, grad);
}

// A wave keeps the rows and positions of its chunk and of as many entries
// after it in its lanes (a chunk is at most 32 long), so that the addresses of
// a batch are known without a load and all of a batch's loads, of dout and of
// the gradient's rows where a run ends, are in flight together.
// STREAM: dout is read past the caches.
template <int ACT, int GRAD, int VEC, bool ACC, bool STREAM>
__global__ void __launch_bounds__(kWaves * 64)
sum_runs(EmbeddingArgs a, EmbeddingWork w, int slabs, int tasks, const void *dout, void *grad)
{
    constexpr int AHEAD = 8;
    const int task = int(blockIdx.x) * kWaves + wave_of();
    const int lane = int(threadIdx.x) % 64;
    const CONSTANT int32_t *begin = (const CONSTANT int32_t *)w.begin;
    if (task >= tasks) {
        // beyond the chunks: rows without a position
        const int z = task - (tasks + kWaves - 1) / kWaves * kWaves;
        if (!ACC && z >= 0) fill_row<GRAD, VEC>(a, w, slabs, z, 0, grad);
        return;
    }
    const int chunk = task / slabs;
    const Columns<VEC> c(task - chunk * slabs, lane, a.width);
    const int valid = begin[a.n_rows];
    const int i0 = chunk * w.chunk;
    if (i0 >= valid) return;
    const int at = min(i0 + lane, valid - 1);
    const int my_row = ((const GLOBAL int32_t *)w.row)[at];
    const int my_pos = ((const GLOBAL int32_t *)w.pos)[at];
    const int my_begin = ((const GLOBAL int32_t *)w.begin)[my_row];
    const int my_end = ((const GLOBAL int32_t *)w.begin)[my_row + 1];

    // entries [begin_at, end) of the lanes, the runs' last ones, and those whose sum
    // goes to a slot
    const int border = min(w.chunk, valid - i0);
    uint64_t last = __ballot(i0 + lane == my_end - 1);
    uint64_t to_more = 0, to_first = 0;
    int begin_at = 0, end = border;
    const int head_begin = __builtin_amdgcn_readlane(my_begin, 0), head_end = __builtin_amdgcn_readlane(my_end, 0);
    if (head_begin < i0) {   // goes on from an earlier chunk: ours if it is long, that chunk's if not
        const int stop = min(head_end - i0, border);
        if (head_end - head_begin > w.chunk)
            to_more = uint64_t(1) << (stop - 1);
        else
            begin_at = stop;
    }
    const int tail_begin = __builtin_amdgcn_readlane(my_begin, border - 1);
    const int tail_end = __builtin_amdgcn_readlane(my_end, border - 1);
    if (tail_begin >= i0 && tail_end > i0 + border) {   // begins here, goes on into the next chunk
        if (tail_end - tail_begin > w.chunk)
            to_first = uint64_t(1) << (border - 1);
        else
            end = tail_end - i0;
    }
    last |= to_more | to_first;

    // the padding row's positions are sorted like any other's and left out
    // here: at most one stretch [skip, resume) of the entries
    const uint64_t pads = __ballot(my_row == w.pad_row && i0 + lane < valid);
    const int skip = pads ? __ffsll((unsigned long long)pads) - 1 : 64, resume = pads ? 64 - __clzll(pads) : 64;

    float sum[VEC] = {};
    const uint64_t rows = last & ~(to_more | to_first);
    for (int part = 0; part < 2; ++part) {
        const int stop = part ? end : min(end, skip);
        for (int e = part ? max(begin_at, resume) : begin_at; e < stop; e += AHEAD) {
            typename Raw<ACT, VEC>::type x[AHEAD];
            typename Raw<GRAD, VEC>::type old[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int64_t pos = __builtin_amdgcn_readlane(my_pos, min(e + k, stop - 1));
                x[k] = load<ACT, VEC, STREAM>(dout, pos * a.act_stride + c.col);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (ACC && e + k < stop && (rows >> (e + k)) & 1) {
                    const int64_t row = __builtin_amdgcn_readlane(my_row, e + k);
                    old[k] = load<GRAD, VEC>(grad, row * a.grad_stride + c.col);
                }
            }
            // All of the batch's loads are waited for here, once. Left to
            // itself the compiler waits where each value is used, which is
            // after the stores of the runs before it, and a wait for a load
            // there waits for those stores too.
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                arrive(x[k]);
                if (ACC) arrive(old[k]);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (e + k < stop) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) sum[j] = __fadd_rn(sum[j], widen<ACT>(x[k][j]));
                    const uint64_t here = uint64_t(1) << (e + k);
                    if (last & here) {
                        if ((to_more | to_first) & here) {
                            float *slot = (to_more & here ? w.more : w.first) + int64_t(chunk) * w.pitch;
                            if (c.on) store<DDP_F32, VEC, false>(slot, c.col, sum, c.skip);   // the join reads it
                        } else {
                            put<GRAD, VEC, ACC>(a, grad, __builtin_amdgcn_readlane(my_row, e + k), c, old[k], sum);
                        }
#pragma unroll
                        for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- join
// A workgroup looks after the long runs that begin in kJoinChunks chunks, over
// a slab of columns. Runs of few pieces go one to a wave; the pieces of one of
// many are split over the waves and the waves' sums added in order. 16 waves
// and 16 chunks: 65536 positions of 64 columns 6.5 us, of two tokens alone 15.6;
// with 4 waves and 8 chunks 11.1 and 34, but where there is little to join 0.3
// to 1.6 us less.
constexpr int kJoinChunks = 16, kJoinWaves = 16;
constexpr int kFewPieces = 16;

// Pieces [k, to) of a long run.
template <int VEC>
__device__ __forceinline__ void add_pieces(const EmbeddingWork &w, const Columns<VEC> &c, int k, int to,
                                           float (&sum)[VEC])
{
    constexpr int AHEAD = 8;
    for (; k < to; k += AHEAD) {
        typename Raw<DDP_F32, VEC>::type x[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) x[j] = load<DDP_F32, VEC>(w.more + int64_t(min(k + j, to - 1)) * w.pitch, c.col);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (k + j < to) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum[e] = __fadd_rn(sum[e], x[j][e]);
            }
    }
}

template <int GRAD, int VEC, bool ACC>
__global__ void __launch_bounds__(kJoinWaves * 64) join_runs(EmbeddingArgs a, EmbeddingWork w, int slabs, void *grad)
{
    __shared__ float part[kJoinWaves][VEC][64];
    const int group = int(blockIdx.x) / slabs, slab = int(blockIdx.x) - group * slabs;
    const int wave = wave_of(), lane = int(threadIdx.x) % 64;
    const CONSTANT int32_t *begin = (const CONSTANT int32_t *)w.begin;
    const int valid = begin[a.n_rows];
    // lane k looks at chunk k of the group
    const int chunk = group * kJoinChunks + lane, i0 = chunk * w.chunk, border = i0 + w.chunk;
    int row = 0, pieces = 0;
    if (lane < kJoinChunks && chunk < w.n_chunks && border < valid) {
        row = ((const GLOBAL int32_t *)w.row)[border - 1];
        const int b = ((const GLOBAL int32_t *)w.begin)[row], e = ((const GLOBAL int32_t *)w.begin)[row + 1];
        if (row != w.pad_row && b >= i0 && e > border && e - b > w.chunk) pieces = (e - 1) / w.chunk - chunk;   // after the first
    }
    uint64_t few = __ballot(pieces > 0 && pieces <= kFewPieces), many = __ballot(pieces > kFewPieces);
    if ((few | many) == 0) return;
    const Columns<VEC> c(slab, lane, a.width);

    for (; many; many &= many - 1) {
        const int k = __ffsll((unsigned long long)many) - 1;
        const int n = __builtin_amdgcn_readlane(pieces, k), first = group * kJoinChunks + k;
        const int64_t r = __builtin_amdgcn_readlane(row, k);
        const int each = (n + kJoinWaves - 1) / kJoinWaves;
        float sum[VEC] = {};
        add_pieces<VEC>(w, c, first + 1 + wave * each, min(first + 1 + n, first + 1 + (wave + 1) * each), sum);
#pragma unroll
        for (int e = 0; e < VEC; ++e) part[wave][e][lane] = sum[e];
        __syncthreads();
        if (wave == 0) {
            typename Raw<GRAD, VEC>::type old;
            if (ACC) old = load<GRAD, VEC>(grad, r * a.grad_stride + c.col);
            const typename Raw<DDP_F32, VEC>::type x = load<DDP_F32, VEC>(w.first + int64_t(first) * w.pitch, c.col);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                sum[e] = x[e];
#pragma unroll
                for (int v = 0; v < kJoinWaves; ++v) sum[e] = __fadd_rn(sum[e], part[v][e][lane]);
            }
            put<GRAD, VEC, ACC>(a, grad, int(r), c, old, sum);
        }
        __syncthreads();
    }
    for (int turn = 0; few; few &= few - 1, ++turn) {
        if (turn % kJoinWaves != wave) continue;
        const int k = __ffsll((unsigned long long)few) - 1;
        const int n = __builtin_amdgcn_readlane(pieces, k), first = group * kJoinChunks + k;
        const int64_t r = __builtin_amdgcn_readlane(row, k);
        typename Raw<GRAD, VEC>::type old;
        if (ACC) old = load<GRAD, VEC>(grad, r * a.grad_stride + c.col);
        const typename Raw<DDP_F32, VEC>::type x = load<DDP_F32, VEC>(w.first + int64_t(first) * w.pitch, c.col);
        float sum[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[e] = x[e];
        add_pieces<VEC>(w, c, first + 1, first + 1 + n, sum);
        put<GRAD, VEC, ACC>(a, grad, int(r), c, old, sum);
    }
}

template <int TABLE, int ACT, int VEC>
hipError_t lookup_vec(EmbeddingArgs a, const void *table, const void *tokens, void *out, hipStream_t s)
{
    const int64_t slabs = slabs_of<VEC>(a.width), all = a.n_tokens;
    // four rows a wave once that leaves every CU sixteen waves
    const bool four = all * slabs >= kLookupRows * 256 * 16;
    const int64_t each = four ? kLookupRows : 1;
    // a launch's grid is limited: kMostWaves of them, then the next launch
    const int64_t most = std::max<int64_t>(1, kMostWaves / slabs) * each;
    const char *tok = static_cast<const char *>(tokens);
    char *dst = static_cast<char *>(out);
    for (int64_t t = 0; t < all; t += most) {
        a.n_tokens = std::min(most, all - t);
        const int64_t tasks = (a.n_tokens + each - 1) / each * slabs;
        const dim3 g(static_cast<unsigned>((tasks + kLookupWaves - 1) / kLookupWaves)), b(kLookupWaves * 64);
        const void *from = tok + t * (a.index64 ? 8 : 4);
        void *to = dst + t * a.act_stride * int64_t(sizeof(typename Raw<ACT, 1>::elem));
        if (four)
            hipLaunchKernelGGL((lookup<TABLE, ACT, VEC, kLookupRows>), g, b, 0, s, a, int(slabs), table, from, to);
        else
            hipLaunchKernelGGL((lookup<TABLE, ACT, VEC, 1>), g, b, 0, s, a, int(slabs), table, from, to);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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

template <class INDEX>
void sort_types(const EmbeddingArgs &a, const EmbeddingWork &w, const INDEX *tokens, dim3 g, dim3 b, unsigned lds,
                hipStream_t s)
{
    const bool one = w.sort_rows <= kSortThreads;   // a thread has one row's counters, or two
    const bool held = w.splits == 1 && a.n_tokens > 0 && a.n_tokens <= int64_t(kSortAhead) * kSortThreads;
    if (one && held)
        hipLaunchKernelGGL((sort_tokens<INDEX, 1, true>), g, b, lds, s, a, w, tokens);
    else if (one)
        hipLaunchKernelGGL((sort_tokens<INDEX, 1, false>), g, b, lds, s, a, w, tokens);
    else
        hipLaunchKernelGGL((sort_tokens<INDEX, 2, false>), g, b, lds, s, a, w, tokens);
}

template <int ACT, int GRAD, int VEC, bool STREAM>
hipError_t sum_vec(const EmbeddingArgs &a, const void *dout, void *grad, bool accumulate, const EmbeddingWork &w,
                   hipStream_t s)
{
    const int64_t slabs = slabs_of<VEC>(a.width);
    const int64_t tasks = w.n_chunks * slabs;
    // the rows that are filled: by the same launch, or, as a launch's grid is
    // limited, by further ones
    const bool beside = !accumulate && a.n_rows * slabs <= kMostWaves;
    if (!accumulate && !beside) {
        const int64_t most = std::max<int64_t>(1, kMostWaves / slabs);
        for (int64_t from = 0; from < a.n_rows; from += most) {
            const int64_t z = std::min(most, a.n_rows - from) * slabs;
            const dim3 g(static_cast<unsigned>((z + kWaves - 1) / kWaves)), b(kWaves * 64);
            hipLaunchKernelGGL((fill_rows<GRAD, VEC>), g, b, 0, s, a, w, int(slabs), int(z), from, grad);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    const int64_t fill = beside ? a.n_rows * slabs : 0;
    const int64_t blocks = (tasks + kWaves - 1) / kWaves + (fill + kWaves - 1) / kWaves;
    if (blocks == 0) return hipSuccess;
    const dim3 g(static_cast<unsigned>(blocks)), b(kWaves * 64);
    if (accumulate)
        hipLaunchKernelGGL((sum_runs<ACT, GRAD, VEC, true, STREAM>), g, b, 0, s, a, w, int(slabs), int(tasks), dout,
                           grad);
    else
        hipLaunchKernelGGL((sum_runs<ACT, GRAD, VEC, false, STREAM>), g, b, 0, s, a, w, int(slabs), int(tasks), dout,
                           grad);
    return hipGetLastError();
}

template <int ACT, int GRAD>
hipError_t sum_types(const EmbeddingArgs &a, const void *dout, void *grad, bool accumulate, const EmbeddingWork &w,
                     hipStream_t s)
{
    constexpr int VEC = sum_vector(ACT, GRAD);
    if (a.width < VEC) return sum_vec<ACT, GRAD, 1, false>(a, dout, grad, accumulate, w, s);
    return w.stream ? sum_vec<ACT, GRAD, VEC, true>(a, dout, grad, accumulate, w, s)
                    : sum_vec<ACT, GRAD, VEC, false>(a, dout, grad, accumulate, w, s);
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

template <int GRAD, int VEC>
hipError_t join_vec(const EmbeddingArgs &a, void *grad, bool accumulate, const EmbeddingWork &w, hipStream_t s)
{
    const int64_t slabs = slabs_of<VEC>(a.width);
    const dim3 g(static_cast<unsigned>((w.n_chunks + kJoinChunks - 1) / kJoinChunks * slabs)), b(kJoinWaves * 64);
    if (accumulate)
        hipLaunchKernelGGL((join_runs<GRAD, VEC, true>), g, b, 0, s, a, w, int(slabs), grad);
    else
        hipLaunchKernelGGL((join_runs<GRAD, VEC, false>), g, b, 0, s, a, w, int(slabs), grad);
    return hipGetLastError();
}

template <int GRAD>
hipError_t join_grad(const EmbeddingArgs &a, void *grad, bool accumulate, const EmbeddingWork &w, hipStream_t s)
{
    return a.width >= 4 ? join_vec<GRAD, 4>(a, grad, accumulate, w, s) : join_vec<GRAD, 1>(a, grad, accumulate, w, s);
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
    const int64_t groups = (a.n_rows + w.sort_rows - 1) / w.sort_rows * w.splits;
    const unsigned lds = unsigned(w.sort_rows) * (kSortWaves + 2) * sizeof(uint32_t);
    const dim3 g(static_cast<unsigned>(groups)), b(kSortThreads);
    if (a.index64)
        sort_types(a, w, static_cast<const int64_t *>(tokens), g, b, lds, s);
    else
        sort_types(a, w, static_cast<const int32_t *>(tokens), g, b, lds, s);
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
