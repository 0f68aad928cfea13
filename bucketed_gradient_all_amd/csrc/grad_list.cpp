// Host half of the gradient lists: validation, the tile tables, and the
// launches of the norm and of clipping.
#include "grad_list.h"
#include "host_common.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <memory>
#include <vector>

using ddp::fail;
using ddp::GradSeg;
using ddp::GradTables;
using ddp::guarded;
using ddp::hip_fail;
using ddp::kGradTile;

namespace {

// Addresses [lo, hi).
struct Span {
    uintptr_t lo, hi;
};

// Sorted and apart.
using Spans = std::vector<Span>;

bool meets(const Spans &v, uintptr_t lo, uintptr_t hi)
{
    const auto it = std::partition_point(v.begin(), v.end(), [lo](const Span &s) { return s.hi <= lo; });
    return it != v.end() && it->lo < hi;
}

}  // namespace

struct ddp_grads {
    GradTables tables{};
    Spans held;      // the tables and the gradients
    Spans written;   // what clipping writes: the gradients in place, or the other buffers
    int device = -1;
    int blocks = 1;        // workgroups of the norm's pass
    int clip_blocks = 1;   // workgroups of the clipping pass
    bool small = false;    // one workgroup clips it
    bool parts = false;    // clipping runs a workgroup a part of a tile, the norm finished before
};

namespace {

constexpr size_t kAlign = 16;

// Tiles of a list, at most: 2^41 elements.
constexpr int64_t kMostTiles = int64_t(1) << 28;

// Tiles of a list that is clipped by a workgroup a part of a tile, at most: a
// launch's grid holds 2^32 threads.
constexpr int64_t kMostPartTiles = int64_t(1) << 21;

size_t align_up(size_t x)
{
    return (x + kAlign - 1) / kAlign * kAlign;
}

int element_size(int32_t type)
{
    return type == DDP_F32 ? 4 : 2;
}

bool known_type(int32_t type)
{
    return type == DDP_F32 || type == DDP_BF16 || type == DDP_F16;
}

int32_t type_of(const ddp_grads_desc &d, int32_t i)
{
    return d.dtype ? d.dtype[i] : int32_t(DDP_F32);
}

int32_t out_type_of(const ddp_grads_desc &d, int32_t i)
{
    return d.out && d.out_dtype ? d.out_dtype[i] : type_of(d, i);
}

// Everything of a desc but its pointers' values.
int check_sizes(const ddp_grads_desc *d)
{
    if (!d) return fail(DDP_ERR_INVALID, "desc is NULL");
    if (d->n_tensors < 0 || d->n_copies < 1)
        return fail(DDP_ERR_INVALID, "a gradient list needs n_tensors >= 0 and n_copies >= 1");
    if (d->n_tensors > 0 && !d->numel) return fail(DDP_ERR_INVALID, "numel is NULL");
    if (!d->out && d->out_dtype) return fail(DDP_ERR_INVALID, "out_dtype is given without out");
    int64_t tiles = 0;
    for (int32_t i = 0; i < d->n_tensors; ++i) {
        if (d->numel[i] < 0 || d->numel[i] > (std::numeric_limits<int64_t>::max() >> 4))
            return fail(DDP_ERR_INVALID, "gradient " + std::to_string(i) + " has a bad size");
        if (!known_type(type_of(*d, i)) || !known_type(out_type_of(*d, i)))
            return fail(DDP_ERR_INVALID, "gradient " + std::to_string(i) + " has an unknown type");
        if (d->numel[i] > 0) tiles += d->numel[i] / kGradTile + 2;   // at most; the cut shifts them
        if (tiles > kMostTiles / d->n_copies)
            return fail(DDP_ERR_INVALID, "the list has too many elements");
    }
    if (int64_t(d->n_tensors) * d->n_copies > std::numeric_limits<int32_t>::max())
        return fail(DDP_ERR_INVALID, "the list has too many tensors");
    return DDP_OK;
}

// Bytes the tables of a valid desc take at most, wherever its tensors lie.
size_t table_bytes(const ddp_grads_desc &d)
{
    size_t segs = 0, tiles = 0;
    for (int32_t i = 0; i < d.n_tensors; ++i)
        if (d.numel[i] > 0) {
            ++segs;
            tiles += size_t(d.numel[i] / kGradTile) + 2;
        }
    const size_t n = size_t(d.n_copies);
    return align_up(n * segs * sizeof(GradSeg)) + align_up(n * tiles * sizeof(int32_t)) + kAlign;
}

struct Range {
    uintptr_t lo, hi;
    int32_t what;   // tensor index for the message, or -1: the workspace
    bool out;       // another buffer that clipping writes
};

int check_overlap(std::vector<Range> &v)
{
    std::sort(v.begin(), v.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    for (size_t i = 1; i < v.size(); ++i)
        if (v[i].lo < v[i - 1].hi) {
            if (v[i].what < 0 || v[i - 1].what < 0)
                return fail(DDP_ERR_INVALID, "the workspace and gradient " +
                                                 std::to_string(std::max(v[i].what, v[i - 1].what)) + " overlap");
            return fail(DDP_ERR_INVALID, "gradients " + std::to_string(v[i - 1].what) + " and " +
                                             std::to_string(v[i].what) + " of the list overlap");
        }
    return DDP_OK;
}

// Those of the sorted ranges that `of` picks; touching ones become one.
template <class F>
Spans spans_of(const std::vector<Range> &v, F of)
{
    Spans s;
    for (const Range &r : v) {
        if (!of(r)) continue;
        if (!s.empty() && s.back().hi == r.lo)
            s.back().hi = r.hi;
        else
            s.push_back({r.lo, r.hi});
    }
    s.shrink_to_fit();
    return s;
}

int create(const ddp_grads_desc *d, ddp_grads **out)
{
    if (!out) return fail(DDP_ERR_INVALID, "out is NULL");
    int rc = check_sizes(d);
    if (rc != DDP_OK) return rc;
    const int32_t N = d->n_tensors, R = d->n_copies;
    if (N > 0 && !d->grads) return fail(DDP_ERR_INVALID, "grads is NULL");
    const size_t need = table_bytes(*d);
    if (!d->workspace || d->workspace_bytes < need || reinterpret_cast<uintptr_t>(d->workspace) % kAlign)
        return fail(DDP_ERR_INVALID,
                    "workspace missing, misaligned or smaller than " + std::to_string(need) + " bytes");
    std::vector<GradSeg> segs;
    std::vector<int32_t> tile_seg;
    const uintptr_t at = reinterpret_cast<uintptr_t>(d->workspace);
    std::vector<Range> ranges{{at, at + need, -1, false}};
    int32_t norm_tiles = 0;
    for (int32_t r = 0; r < R; ++r) {
        for (int32_t i = 0; i < N; ++i) {
            const int64_t n = d->numel[i];
            if (n == 0) continue;
            const size_t k = size_t(r) * size_t(N) + size_t(i);
            GradSeg s{};
            s.in = uint8_t(type_of(*d, i));
            s.out = uint8_t(out_type_of(*d, i));
            s.src = d->grads[k];
            s.dst = d->out ? d->out[k] : const_cast<void *>(s.src);
            s.len = n;
            const uintptr_t src = reinterpret_cast<uintptr_t>(s.src), dst = reinterpret_cast<uintptr_t>(s.dst);
            const uintptr_t isz = uintptr_t(element_size(s.in)), osz = uintptr_t(element_size(s.out));
            if (!src || !dst) return fail(DDP_ERR_INVALID, "gradient " + std::to_string(i) + " has a NULL pointer");
            if (src % isz || dst % osz)
                return fail(DDP_ERR_INVALID, "gradient " + std::to_string(i) + " is misaligned for its type");
            ranges.push_back({src, src + isz * uintptr_t(n), i, false});
            if (d->out) ranges.push_back({dst, dst + osz * uintptr_t(n), i, true});
            s.shift = int16_t(dst % 256 / osz);
            s.tile0 = int32_t(tile_seg.size());
            const int64_t tiles = (n + s.shift + kGradTile - 1) / kGradTile;
            tile_seg.insert(tile_seg.end(), size_t(tiles), int32_t(segs.size()));
            segs.push_back(s);
        }
        if (r == 0) norm_tiles = int32_t(tile_seg.size());
    }
    rc = check_overlap(ranges);
    if (rc != DDP_OK) return rc;

    std::unique_ptr<ddp_grads> g(new ddp_grads());
    g->held = spans_of(ranges, [](const Range &r) { return !r.out; });
    g->written = spans_of(ranges, [d](const Range &r) { return r.what >= 0 && r.out == (d->out != nullptr); });
    hipError_t e = hipGetDevice(&g->device);
    int cus = 0;
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, g->device);
    if (e != hipSuccess) return hip_fail("device of the gradient list", e);
    const size_t segs_bytes = align_up(segs.size() * sizeof(GradSeg));
    std::vector<uint8_t> host(segs_bytes + tile_seg.size() * sizeof(int32_t));
    if (!segs.empty()) {
        std::memcpy(host.data(), segs.data(), segs.size() * sizeof(GradSeg));
        std::memcpy(host.data() + segs_bytes, tile_seg.data(), tile_seg.size() * sizeof(int32_t));
        e = hipMemcpy(d->workspace, host.data(), host.size(), hipMemcpyHostToDevice);
        if (e != hipSuccess) return hip_fail("workspace upload", e);
    }
    uint8_t *ws = static_cast<uint8_t *>(d->workspace);
    g->tables.segs = reinterpret_cast<const GradSeg *>(ws);
    g->tables.tile_seg = reinterpret_cast<const int32_t *>(ws + segs_bytes);
    g->tables.norm_tiles = norm_tiles;
    g->tables.all_tiles = int32_t(tile_seg.size());
    g->tables.in_place = d->out == nullptr;
    g->small = g->tables.all_tiles <= ddp::kSmallClip;
    // workgroups that go from tile to tile, as many as fill the chip. The norm
    // does best with four a CU (953M bf16 elements 285 us, eight 294, two 292)
    // and leaves as many partials. Clipping takes eight: of two, four, eight,
    // sixteen and thirty-two 335M fp32 elements in place take 476, 499, 496,
    // 490 and 486 us to scale, 203 to 213 with the norm if they lie below the
    // bound, and 30M into another buffer 61 to 63.
    g->blocks = std::max(1, std::min({norm_tiles, ddp::kMaxPartials, 4 * cus}));
    g->clip_blocks = std::max(1, std::min(g->tables.all_tiles, 8 * cus));
    // Into other buffers every tensor is written, so a workgroup a part of a
    // tile pays. In place there is mostly nothing to do but to see that the
    // norm is below the bound, which 2048 workgroups do in 5 us; 41116, one a
    // tile, took 11. The price: where they do scale, 335M fp32 elements on
    // eight replicas take 4.14 ms (5.2 TB/s) against 3.58 (6.0 TB/s) with a
    // workgroup a part.
    g->parts = !g->tables.in_place && g->tables.all_tiles > ddp::kManyTiles && g->tables.all_tiles <= kMostPartTiles;
    *out = g.release();
    return DDP_OK;
}

// A call's device: the list's must be current, and the stream must be its.
int check_device(const ddp_grads *g, hipStream_t s)
{
    int now = -1;
    hipError_t e = hipGetDevice(&now);
    if (e != hipSuccess) return hip_fail("current device", e);
    if (now != g->device)
        return fail(DDP_ERR_INVALID, "the gradient list is on device " + std::to_string(g->device) +
                                         ", the current device is " + std::to_string(now));
    return ddp::check_stream(s, now);
}

// What a call writes must lie apart from what it reads, of the other workgroups
// too: partial sums over the tables would send them anywhere.
int check_apart(const ddp_grads *g, const char *what, uintptr_t lo, size_t bytes, bool clips)
{
    if (meets(g->held, lo, lo + bytes) || (clips && meets(g->written, lo, lo + bytes)))
        return fail(DDP_ERR_INVALID, std::string(what) + " overlaps a tensor or the workspace of the gradient list");
    return DDP_OK;
}

int check_call(const ddp_grads *g, int32_t norm_type, const float *norm, const void *scratch, size_t scratch_bytes,
               bool clips, hipStream_t s)
{
    if (!g) return fail(DDP_ERR_INVALID, "the gradient list is NULL");
    if (norm_type != DDP_NORM_INF && norm_type != DDP_NORM_L1 && norm_type != DDP_NORM_L2)
        return fail(DDP_ERR_INVALID, "unknown norm " + std::to_string(norm_type));
    if (!norm || reinterpret_cast<uintptr_t>(norm) % 4)
        return fail(DDP_ERR_INVALID, "norm is NULL or misaligned");
    const size_t need = sizeof(double) * size_t(g->blocks);
    if (!scratch || scratch_bytes < need || reinterpret_cast<uintptr_t>(scratch) % 8)
        return fail(DDP_ERR_INVALID,
                    "scratch missing, misaligned or smaller than " + std::to_string(need) + " bytes");
    // the first workgroup of the clipping pass writes the norm while others
    // still read the partials
    const uintptr_t to = reinterpret_cast<uintptr_t>(norm), from = reinterpret_cast<uintptr_t>(scratch);
    if (to + sizeof(float) > from && to < from + need)
        return fail(DDP_ERR_INVALID, "norm lies inside the scratch");
    int rc = check_apart(g, "norm", to, sizeof(float), clips);
    if (rc == DDP_OK) rc = check_apart(g, "scratch", from, need, clips);
    return rc == DDP_OK ? check_device(g, s) : rc;
}

int check_max_norm(float max_norm)
{
    if (!(max_norm >= 0.0f) || std::isinf(max_norm))
        return fail(DDP_ERR_INVALID, "max_norm must be finite and not negative");
    return DDP_OK;
}

// The desc of a reducer's results, with the arrays it points to.
struct ReducerDesc {
    std::vector<int64_t> numel;
    std::vector<const void *> ptrs;
    ddp_grads_desc d{};
    int device = -1;
};

int reducer_desc(const ddp_reducer *r, ReducerDesc &out)
{
    if (!r) return fail(DDP_ERR_INVALID, "reducer is NULL");
    const ddp::ReducerBuffers b = ddp::reducer_buffers(r);
    if (!b.flat) return fail(DDP_ERR_INVALID, "reducer has no device");
    out.device = b.device;
    if (b.reduce_scatter) {
        for (int32_t k = 0; k < b.n_buckets; ++k) {
            const int64_t n = b.bucket_bytes[k] / 4;
            const int64_t q = n / b.world + (n % b.world != 0);
            for (int32_t c = 0; c < b.world && q > 0; ++c) {
                const int64_t lo = std::min(n, c * q), hi = std::min(n, lo + q);
                if (lo == hi) break;
                out.numel.push_back(hi - lo);
                out.ptrs.push_back(b.flat[c] + b.bucket_flat[k] / 4 + lo);
            }
        }
        out.d.n_copies = 1;
    } else {
        int64_t n = 0;
        for (int32_t k = 0; k < b.n_buckets; ++k) n += b.bucket_bytes[k] / 4;
        out.numel.push_back(n);
        out.ptrs.assign(b.flat, b.flat + b.world);
        out.d.n_copies = b.world;
    }
    if (out.numel.size() > size_t(std::numeric_limits<int32_t>::max()))
        return fail(DDP_ERR_INVALID, "the list has too many tensors");
    out.d.n_tensors = int32_t(out.numel.size());
    out.d.numel = out.numel.data();
    out.d.grads = out.ptrs.data();
    return DDP_OK;
}

}  // namespace

namespace ddp {

int check_stream(hipStream_t s, int device)
{
    // the null and the per-thread stream are the current device's (and the
    // second is no object that could be asked)
    if (!s || s == hipStreamPerThread) return DDP_OK;
    hipDevice_t of = -1;
    const hipError_t e = hipStreamGetDevice(s, &of);
    if (e != hipSuccess) return hip_fail("device of the stream", e);
    if (of != device)
        return fail(DDP_ERR_INVALID, "the stream belongs to device " + std::to_string(of) +
                                         ", the current device is " + std::to_string(device));
    return DDP_OK;
}

}  // namespace ddp

extern "C" {

size_t ddp_grads_workspace_bytes(const ddp_grads_desc *desc)
{
    size_t n = 0;
    guarded([&] {
        const int rc = check_sizes(desc);
        if (rc == DDP_OK) n = table_bytes(*desc);
        return rc;
    });
    return n;
}

int ddp_grads_create(const ddp_grads_desc *desc, ddp_grads **out)
{
    return guarded([&] { return create(desc, out); });
}

size_t ddp_reducer_grads_workspace_bytes(const ddp_reducer *r)
{
    size_t n = 0;
    guarded([&] {
        ReducerDesc d;
        const int rc = reducer_desc(r, d);
        if (rc != DDP_OK) return rc;
        n = ddp_grads_workspace_bytes(&d.d);
        return int(DDP_OK);
    });
    return n;
}

int ddp_grads_from_reducer(const ddp_reducer *r, void *workspace, size_t workspace_bytes, ddp_grads **out)
{
    return guarded([&] {
        ReducerDesc d;
        const int rc = reducer_desc(r, d);
        if (rc != DDP_OK) return rc;
        // the list will launch on the device that is current now
        int now = -1;
        const hipError_t e = hipGetDevice(&now);
        if (e != hipSuccess) return hip_fail("current device", e);
        if (now != d.device)
            return fail(DDP_ERR_INVALID, "the reducer is on device " + std::to_string(d.device) +
                                             ", the current device is " + std::to_string(now));
        d.d.workspace = workspace;
        d.d.workspace_bytes = workspace_bytes;
        return create(&d.d, out);
    });
}

int ddp_grads_destroy(ddp_grads *g)
{
    delete g;
    return DDP_OK;
}

int ddp_grads_scratch_bytes(const ddp_grads *g, size_t *bytes)
{
    return guarded([&] {
        if (!g || !bytes) return fail(DDP_ERR_INVALID, "NULL argument");
        *bytes = sizeof(double) * size_t(g->blocks);
        return int(DDP_OK);
    });
}

int ddp_grad_norm(const ddp_grads *g, int32_t norm_type, float *norm, void *scratch, size_t scratch_bytes,
                  void *stream)
{
    return guarded([&] {
        const hipStream_t s = ddp::stream_of(stream);
        const int rc = check_call(g, norm_type, norm, scratch, scratch_bytes, false, s);
        if (rc != DDP_OK) return rc;
        hipError_t e;
        if (g->tables.norm_tiles <= ddp::kSmallNorm) {
            e = ddp::launch_small(norm_type, g->tables, false, 0.0f, norm, s);
        } else {
            e = ddp::launch_norm_partials(norm_type, g->tables, g->blocks, scratch, s);
            if (e == hipSuccess) e = ddp::launch_norm_finish(norm_type, g->blocks, scratch, norm, s);
        }
        return e == hipSuccess ? int(DDP_OK) : hip_fail("gradient norm", e);
    });
}

int ddp_clip_grad_norm(const ddp_grads *g, int32_t norm_type, float max_norm, float *norm, void *scratch,
                       size_t scratch_bytes, void *stream)
{
    return guarded([&] {
        const hipStream_t s = ddp::stream_of(stream);
        int rc = check_call(g, norm_type, norm, scratch, scratch_bytes, true, s);
        if (rc == DDP_OK) rc = check_max_norm(max_norm);
        if (rc != DDP_OK) return rc;
        hipError_t e;
        if (g->small) {
            e = ddp::launch_small(norm_type, g->tables, true, max_norm, norm, s);
        } else {
            e = ddp::launch_norm_partials(norm_type, g->tables, g->blocks, scratch, s);
            if (e == hipSuccess && g->parts) {
                e = ddp::launch_norm_finish(norm_type, g->blocks, scratch, norm, s);
                if (e == hipSuccess) e = ddp::launch_clip_parts(g->tables, {max_norm, norm}, s);
            } else if (e == hipSuccess) {
                e = ddp::launch_clip(norm_type, g->tables, g->clip_blocks, {max_norm, nullptr}, g->blocks, scratch,
                                     norm, s);
            }
        }
        return e == hipSuccess ? int(DDP_OK) : hip_fail("gradient clipping", e);
    });
}

int ddp_clip_grads(const ddp_grads *g, float max_norm, const float *norm, void *stream)
{
    return guarded([&] {
        const hipStream_t s = ddp::stream_of(stream);
        if (!g) return fail(DDP_ERR_INVALID, "the gradient list is NULL");
        if (!norm || reinterpret_cast<uintptr_t>(norm) % 4)
            return fail(DDP_ERR_INVALID, "norm is NULL or misaligned");
        // every workgroup reads it, while others write already
        const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
        if (meets(g->written, at, at + sizeof(float)))
            return fail(DDP_ERR_INVALID, "norm lies where the call writes");
        int rc = check_max_norm(max_norm);
        if (rc == DDP_OK) rc = check_device(g, s);
        if (rc != DDP_OK) return rc;
        if (g->tables.all_tiles == 0) return int(DDP_OK);
        const hipError_t e = g->parts ? ddp::launch_clip_parts(g->tables, {max_norm, norm}, s)
                                      : ddp::launch_clip(DDP_NORM_L2, g->tables, g->clip_blocks, {max_norm, norm}, 0,
                                                         nullptr, nullptr, s);
        return e == hipSuccess ? int(DDP_OK) : hip_fail("gradient clipping", e);
    });
}

}  // extern "C"
