// Host half of the embedding operators: validation, the workspace's layout
// and the launches.
#include "embedding.h"
#include "host_common.h"
#include "spans.h"

#include <algorithm>
#include <cmath>
#include <limits>

using ddp::EmbeddingArgs;
using ddp::EmbeddingWork;
using ddp::fail;
using ddp::guarded;
using ddp::hip_fail;
using ddp::rows_meet;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxTokens = int64_t(1) << 30;

size_t align_up(size_t x)
{
    return (x + kAlign - 1) / kAlign * kAlign;
}

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

int element_size(int32_t type)
{
    return type == DDP_F32 ? 4 : 2;
}

bool known_type(int32_t type)
{
    return type == DDP_F32 || type == DDP_BF16 || type == DDP_F16;
}

int check_desc(const ddp_embedding_desc *d, int64_t n_tokens)
{
    if (!d) return fail(DDP_ERR_INVALID, "desc is NULL");
    if (d->n_rows < 0 || d->n_rows >= std::numeric_limits<int32_t>::max())
        return fail(DDP_ERR_INVALID, "n_rows must be in [0, 2^31 - 1)");
    if (d->first_row > std::numeric_limits<int64_t>::max() - d->n_rows)
        return fail(DDP_ERR_INVALID, "first_row + n_rows exceeds 2^63 - 1");
    if (d->width < 0 || d->width > std::numeric_limits<int32_t>::max())
        return fail(DDP_ERR_INVALID, "width must be in [0, 2^31)");
    if (d->index_dtype != DDP_I32 && d->index_dtype != DDP_I64)
        return fail(DDP_ERR_INVALID, "unknown index type " + std::to_string(d->index_dtype));
    if (!known_type(d->table_dtype) || !known_type(d->grad_dtype) || !known_type(d->act_dtype))
        return fail(DDP_ERR_INVALID, "unknown element type in the desc");
    // strides up to 2^31 keep every row's offset far inside 64 bits
    const int64_t most = int64_t(1) << 31;
    if (d->table_stride < d->width || d->grad_stride < d->width || d->table_stride > most || d->grad_stride > most)
        return fail(DDP_ERR_INVALID, "table_stride and grad_stride must be in [width, 2^31]");
    if (d->act_stride < 0 || d->act_stride > most)
        return fail(DDP_ERR_INVALID, "act_stride must be in [0, 2^31]");
    if (std::isnan(d->scale)) return fail(DDP_ERR_INVALID, "scale is NaN");
    if (n_tokens < 0 || n_tokens > kMaxTokens) return fail(DDP_ERR_INVALID, "n_tokens must be in [0, 2^30]");
    return DDP_OK;
}

EmbeddingArgs args_of(const ddp_embedding_desc &d, int64_t n_tokens)
{
    EmbeddingArgs a{};
    a.n_rows = d.n_rows;
    a.width = d.width;
    a.first_row = d.first_row;
    a.table_stride = d.table_stride;
    a.grad_stride = d.grad_stride;
    a.act_stride = d.act_stride;
    a.n_tokens = n_tokens;
    a.scale = d.scale;
    a.index64 = d.index_dtype == DDP_I64;
    a.table_dtype = d.table_dtype;
    a.grad_dtype = d.grad_dtype;
    a.act_dtype = d.act_dtype;
    return a;
}

int check_pointer(const char *what, const void *p, int align)
{
    if (!p) return fail(DDP_ERR_INVALID, std::string(what) + " is NULL");
    if (reinterpret_cast<uintptr_t>(p) % uintptr_t(align))
        return fail(DDP_ERR_INVALID, std::string(what) + " is misaligned");
    return DDP_OK;
}

int check_device(hipStream_t s)
{
    int now = -1;
    const hipError_t e = hipGetDevice(&now);
    if (e != hipSuccess) return hip_fail("current device", e);
    return ddp::check_stream(s, now);
}

// Waves that share the positions of the sum, at most, before chunks grow.
constexpr int64_t kWantedWaves = 8192;

// Bytes of dout from which it is read past the caches: well below the 256 MiB
// of the last cache it may still lie there from the kernel that wrote it. 2048
// bf16 columns added to fp32, past the caches against through them: 32 MiB 34.6
// us against 32.8, 64 MiB 49.2 against 48.8, 128 MiB 72.8 against 77.3, 256 MiB
// 116 against 135; with dout written right before (that copy's time taken off),
// 64 MiB 49.4 against 48.1, 128 MiB 72 against 74, 256 MiB 122 against 132.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

// Waves side by side over a row's columns, and of the sum in all, at most:
// what a launch's grid holds, 2^32 threads, with room for the rows that a whole
// gradient fills.
constexpr int64_t kMostSlabs = int64_t(1) << 20, kMostChunkWaves = int64_t(1) << 25;

int64_t slabs_of(const ddp_embedding_desc &d)
{
    return std::max<int64_t>(1, ceil_div(d.width, 64 * ddp::sum_vector(d.act_dtype, d.grad_dtype)));
}

// Positions of a chunk: as many as still leave kWantedWaves waves, 8 to 32.
// Longer chunks cut fewer runs and leave the join less; the waves fill the chip
// (32768 positions of 2048 columns: chunks of 32 55.3 us and the join 5.6, of
// 16 53.1 and 9.8).
int32_t chunk_of(const ddp_embedding_desc &d, int64_t n_tokens)
{
    int32_t c = 8;
    while (c < ddp::kMaxChunk && n_tokens * slabs_of(d) > kWantedWaves * c) c *= 2;
    return c;
}

// Chunks of any call of up to n_tokens positions: shorter calls may have
// shorter chunks, so more of them.
int64_t most_chunks(const ddp_embedding_desc &d, int64_t n_tokens)
{
    const int64_t own = ceil_div(n_tokens, chunk_of(d, n_tokens));
    return std::max(own, std::min(ceil_div(n_tokens, 8), kWantedWaves / slabs_of(d) + 1));
}

struct Layout {
    size_t row, pos, begin, first, more, total;
    int64_t pitch;
};

Layout layout_of(const ddp_embedding_desc &d, int64_t n_tokens)
{
    Layout l{};
    size_t cur = 0;
    const auto take = [&](size_t bytes) {
        const size_t at = cur;
        cur += align_up(bytes);
        return at;
    };
    l.pitch = ceil_div(d.width, 4) * 4;
    const size_t slots = sizeof(float) * size_t(most_chunks(d, n_tokens)) * size_t(l.pitch);
    l.row = take(sizeof(int32_t) * size_t(n_tokens));
    l.pos = take(sizeof(int32_t) * size_t(n_tokens));
    l.begin = take(sizeof(int32_t) * size_t(d.n_rows + 1));
    l.first = take(slots);
    l.more = take(slots);
    l.total = cur;
    return l;
}

// Positions for which another workgroup shares a range's sorting: 32000 rows,
// 8191 positions 9.2 us with one, 9.4 with two, 12.1 with four; 32768 positions
// 21.6, 16.6, 15.0 (eight: 21.2); 262144 positions 67 with four, 60 with eight,
// 58 with sixteen.
constexpr int64_t kSplitTokens = 8192;

// The sort's workgroups: about 256, one a CU, are ranges of rows, as far as a
// range's counters fit the LDS, times the workgroups of a range.
void sort_plan(const ddp_embedding_desc &d, int64_t n, EmbeddingWork *w)
{
    const int64_t fewest = ceil_div(d.n_rows, ddp::kMaxSortRows);   // ranges
    const int64_t splits =
        std::max<int64_t>(1, std::min({int64_t(64), n / kSplitTokens, 256 / std::max<int64_t>(1, fewest)}));
    w->sort_rows =
        int32_t(std::min<int64_t>(ddp::kMaxSortRows, std::max<int64_t>(16, ceil_div(d.n_rows, 256 / splits))));
    w->splits = int32_t(splits);
}

// Bytes of dout that one workgroup of the one-launch path may have to read, if
// all positions have one token.
constexpr int64_t kSmallBytes = int64_t(2) << 20;

// Whether a call takes the one-launch path, and how: about 256 workgroups, or
// up to twice as many if the table's ranges need them. Replayed from a graph,
// one launch against three (30522 rows of 1024 fp32 columns): 128 positions 5.7
// us against 11.6, 1024 7.7 against 13.7, 2048 8.4 against 14.4; called one by
// one the host saves two launches too. The other side of it: 2048 positions of
// one and the same token are one range's, 29 us against 20.
bool small_plan(const ddp_embedding_desc &d, int64_t n, ddp::SmallPlan *p)
{
    const int64_t vec = ddp::sum_vector(d.act_dtype, d.grad_dtype);
    if (n > ddp::kSmallTokens || d.width < vec) return false;
    if (n * 64 * vec * element_size(d.act_dtype) > kSmallBytes) return false;
    const int64_t slabs = slabs_of(d);
    if (slabs > 256) return false;
    const int64_t rows = std::min<int64_t>(ddp::kSmallRows, std::max<int64_t>(16, ceil_div(d.n_rows, 256 / slabs)));
    if (ceil_div(d.n_rows, rows) * slabs > 512) return false;
    p->rows = int32_t(rows);
    p->slabs = int32_t(slabs);
    return true;
}

int32_t pad_row_of(const ddp_embedding_desc &d)
{
    const bool held = d.padding_idx >= 0 && d.padding_idx >= d.first_row &&
                      uint64_t(d.padding_idx) - uint64_t(d.first_row) < uint64_t(d.n_rows);
    return held ? int32_t(d.padding_idx - d.first_row) : -1;
}

int lookup(const ddp_embedding_desc *d, const void *table, const void *tokens, int64_t n, void *out, hipStream_t s)
{
    int rc = check_desc(d, n);
    if (rc != DDP_OK) return rc;
    if (n > 1 && d->act_stride < d->width)
        return fail(DDP_ERR_INVALID, "act_stride must be at least the width for the lookup's output");
    if (n == 0 || d->width == 0) return DDP_OK;
    if (d->n_rows > 0) rc = check_pointer("table", table, element_size(d->table_dtype));
    if (rc == DDP_OK) rc = check_pointer("tokens", tokens, d->index_dtype == DDP_I64 ? 8 : 4);
    if (rc == DDP_OK) rc = check_pointer("out", out, element_size(d->act_dtype));
    if (rc != DDP_OK) return rc;
    if (ceil_div(d->width, 64) > kMostSlabs) return fail(DDP_ERR_INVALID, "width is too large for one call");
    rc = check_device(s);
    if (rc != DDP_OK) return rc;
    const hipError_t e = ddp::launch_lookup(args_of(*d, n), table, tokens, out, s);
    return e == hipSuccess ? DDP_OK : hip_fail("embedding lookup", e);
}

// The sum takes rows and positions from the workspace as they stand there:
// written over, they would be addresses of anything.
int check_workspace_apart(const ddp_embedding_desc &d, const void *dout, const void *tokens, int64_t n, const void *g,
                          const void *workspace, size_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(workspace), hi = lo + bytes;
    const int64_t act = element_size(d.act_dtype), out = element_size(d.grad_dtype);
    const int64_t index = d.index_dtype == DDP_I64 ? 8 : 4;
    if (rows_meet(g, d.n_rows, d.grad_stride * out, d.width * out, lo, hi))
        return fail(DDP_ERR_INVALID, "the workspace and grad overlap");
    if (rows_meet(dout, n, d.act_stride * act, d.width * act, lo, hi))
        return fail(DDP_ERR_INVALID, "the workspace and dout overlap");
    if (rows_meet(tokens, n, index, index, lo, hi)) return fail(DDP_ERR_INVALID, "the workspace and tokens overlap");
    return DDP_OK;
}

int grad(const ddp_embedding_desc *d, const void *dout, const void *tokens, int64_t n, void *g, bool accumulate,
         void *workspace, size_t workspace_bytes, hipStream_t s)
{
    int rc = check_desc(d, n);
    if (rc != DDP_OK) return rc;
    if (d->n_rows == 0 || d->width == 0 || (n == 0 && accumulate)) return DDP_OK;
    if (n > 0) rc = check_pointer("dout", dout, element_size(d->act_dtype));
    if (rc == DDP_OK && n > 0) rc = check_pointer("tokens", tokens, d->index_dtype == DDP_I64 ? 8 : 4);
    if (rc == DDP_OK) rc = check_pointer("grad", g, element_size(d->grad_dtype));
    if (rc != DDP_OK) return rc;
    const Layout l = layout_of(*d, n);
    if (!workspace || workspace_bytes < l.total || reinterpret_cast<uintptr_t>(workspace) % kAlign)
        return fail(DDP_ERR_INVALID,
                    "workspace missing, misaligned or smaller than " + std::to_string(l.total) + " bytes");
    EmbeddingWork w{};
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    w.row = reinterpret_cast<int32_t *>(ws + l.row);
    w.pos = reinterpret_cast<int32_t *>(ws + l.pos);
    w.begin = reinterpret_cast<int32_t *>(ws + l.begin);
    w.first = reinterpret_cast<float *>(ws + l.first);
    w.more = reinterpret_cast<float *>(ws + l.more);
    w.pitch = l.pitch;
    w.chunk = chunk_of(*d, n);
    w.n_chunks = int32_t(ceil_div(n, w.chunk));
    sort_plan(*d, n, &w);
    w.stream = n > kStreamBytes / (d->width * element_size(d->act_dtype));
    w.pad_row = pad_row_of(*d);
    const int64_t wide = ceil_div(d->width, 64);   // slabs of the narrowest kernel, an upper bound
    if (wide > kMostSlabs || w.n_chunks * wide > kMostChunkWaves)
        return fail(DDP_ERR_INVALID, "n_tokens times width is too large for one call");
    rc = check_workspace_apart(*d, dout, tokens, n, g, workspace, l.total);
    if (rc == DDP_OK) rc = check_device(s);
    if (rc != DDP_OK) return rc;
    const EmbeddingArgs a = args_of(*d, n);
    ddp::SmallPlan small{};
    small.pad_row = w.pad_row;
    if (small_plan(*d, n, &small)) {
        const hipError_t e = ddp::launch_small_grad(a, small, tokens, dout, g, accumulate, s);
        return e == hipSuccess ? DDP_OK : hip_fail("embedding gradient", e);
    }
    hipError_t e = ddp::launch_sort(a, tokens, w, s);
    if (e == hipSuccess) e = ddp::launch_sum(a, dout, g, accumulate, w, s);
    // a long run needs more than a chunk's positions
    if (e == hipSuccess && n > w.chunk) e = ddp::launch_join(a, g, accumulate, w, s);
    return e == hipSuccess ? DDP_OK : hip_fail("embedding gradient", e);
}

}  // namespace

extern "C" {

int ddp_embedding_lookup(const ddp_embedding_desc *desc, const void *table, const void *tokens, int64_t n_tokens,
                         void *out, void *stream)
{
    return guarded([&] { return lookup(desc, table, tokens, n_tokens, out, ddp::stream_of(stream)); });
}

size_t ddp_embedding_grad_workspace_bytes(const ddp_embedding_desc *desc, int64_t n_tokens)
{
    size_t n = 0;
    guarded([&] {
        const int rc = check_desc(desc, n_tokens);
        if (rc == DDP_OK) n = layout_of(*desc, n_tokens).total;
        return rc;
    });
    return n;
}

int ddp_embedding_grad(const ddp_embedding_desc *desc, const void *dout, const void *tokens, int64_t n_tokens,
                       void *grad_out, int32_t accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        return grad(desc, dout, tokens, n_tokens, grad_out, accumulate != 0, workspace, workspace_bytes,
                    ddp::stream_of(stream));
    });
}

}  // extern "C"
