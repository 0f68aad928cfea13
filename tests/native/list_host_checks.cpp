// The host half of the gradient lists and the embedding operators against
// stand-ins for the HIP runtime (fake_hip.cpp) and the kernel launchers
// (below), built under AddressSanitizer and UndefinedBehaviorSanitizer. Checks:
//  * a list's uploaded tables cover every element of every copy exactly once,
//    cut at destination addresses that are multiples of 256 bytes, inside the
//    workspace it asked for;
//  * a reducer's list: one tensor a replica after an all-reduce, the owners'
//    chunks after a reduce-scatter;
//  * which launches a call makes, and that a stream of another device is
//    refused before any;
//  * the embedding gradient's workspace: its parts are disjoint, large enough
//    for the chunks of the call, and inside the size for any longer call;
//  * host memory exhaustion gives DDP_ERR_NOMEM and leaks nothing.
#include "ddp.h"
#include "embedding.h"
#include "fake_hip.h"
#include "grad_list.h"

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <random>
#include <string>
#include <vector>

#include "failing_new.h"

namespace {

int g_bad = 0;
int g_stream_device = 0;
std::vector<std::string> g_launches;
ddp::GradTables g_tables;
int g_blocks = 0;
ddp::EmbeddingWork g_work;
ddp::SmallPlan g_small;

void expect(bool ok, const std::string &what)
{
    if (!ok && g_bad++ < 30) std::fprintf(stderr, "FAILED: %s\n", what.c_str());
}

hipError_t note(const char *what)
{
    if (fake::g_logging) g_launches.push_back(what);
    return hipSuccess;
}

}  // namespace

extern "C" hipError_t hipStreamGetDevice(hipStream_t s, hipDevice_t *device)
{
    // the runtime's own ends the process for these
    expect(s && s != hipStreamLegacy && s != hipStreamPerThread, "a special stream handle was asked for its device");
    *device = g_stream_device;
    return hipSuccess;
}

namespace ddp {

hipError_t launch_norm_partials(int, const GradTables &t, int blocks, void *, hipStream_t)
{
    g_tables = t;
    g_blocks = blocks;
    return note("partials");
}
hipError_t launch_norm_finish(int, int, const void *, float *, hipStream_t) { return note("finish"); }
hipError_t launch_clip(int, const GradTables &t, int, const ClipFactor &f, int, const void *, float *, hipStream_t)
{
    g_tables = t;
    return note(f.norm ? "clip given" : "clip");
}
hipError_t launch_clip_parts(const GradTables &t, const ClipFactor &, hipStream_t)
{
    g_tables = t;
    return note("clip parts");
}
hipError_t launch_small(int, const GradTables &t, bool clip, float, float *, hipStream_t)
{
    g_tables = t;
    return note(clip ? "small clip" : "small");
}
hipError_t launch_small_grad(const EmbeddingArgs &, const SmallPlan &p, const void *, const void *, void *, bool,
                             hipStream_t)
{
    g_small = p;
    return note("small grad");
}
hipError_t launch_lookup(const EmbeddingArgs &, const void *, const void *, void *, hipStream_t)
{
    return note("lookup");
}
hipError_t launch_sort(const EmbeddingArgs &, const void *, const EmbeddingWork &w, hipStream_t)
{
    g_work = w;
    return note("sort");
}
hipError_t launch_sum(const EmbeddingArgs &, const void *, void *, bool, const EmbeddingWork &, hipStream_t)
{
    return note("sum");
}
hipError_t launch_join(const EmbeddingArgs &, void *, bool, const EmbeddingWork &, hipStream_t)
{
    return note("join");
}

}  // namespace ddp

namespace {

std::vector<std::string> launches()
{
    std::vector<std::string> v;
    v.swap(g_launches);
    return v;
}

// A workspace at a 256-byte boundary.
struct Space {
    std::vector<uint8_t> store;
    uint8_t *at;
    explicit Space(size_t n) : store(n + 256), at(store.data())
    {
        while (reinterpret_cast<uintptr_t>(at) % 256) ++at;
    }
};

uintptr_t elem(int32_t type)
{
    return type == DDP_F32 ? 4 : 2;
}

void check_tables(const ddp_grads_desc &d, const uint8_t *ws, size_t bytes, const std::string &name)
{
    const ddp::GradTables &t = g_tables;
    const uint8_t *lo = reinterpret_cast<const uint8_t *>(t.segs);
    const uint8_t *hi = reinterpret_cast<const uint8_t *>(t.tile_seg + t.all_tiles);
    expect(lo >= ws && hi <= ws + bytes, name + ": tables outside the workspace");
    int tile = 0;
    for (int r = 0; r < d.n_copies; ++r) {
        for (int i = 0; i < d.n_tensors; ++i) {
            const int64_t n = d.numel[i];
            if (n == 0) continue;
            const size_t k = size_t(r) * d.n_tensors + i;
            const int32_t in = d.dtype ? d.dtype[i] : int32_t(DDP_F32);
            const int32_t out = d.out_dtype ? d.out_dtype[i] : in;
            int64_t done = 0;
            while (done < n) {
                if (tile >= t.all_tiles) {
                    expect(false, name + ": too few tiles");
                    return;
                }
                const ddp::GradSeg &s = t.segs[t.tile_seg[tile]];
                expect(s.src == d.grads[k] && s.dst == (d.out ? d.out[k] : d.grads[k]) && s.len == n &&
                           s.in == in && s.out == out,
                       name + ": wrong record");
                const int64_t base = int64_t(tile - s.tile0) * ddp::kGradTile - s.shift;
                expect(std::max<int64_t>(base, 0) == done, name + ": a gap between tiles");
                expect((reinterpret_cast<uintptr_t>(s.dst) + uintptr_t(base) * elem(out)) % 256 == 0,
                       name + ": a tile is not cut at a line");
                done = std::min(n, base + ddp::kGradTile);
                ++tile;
            }
        }
        if (r == 0) expect(tile == t.norm_tiles, name + ": the norm's tiles");
    }
    expect(tile == t.all_tiles, name + ": tiles left over");
}

void lists()
{
    std::mt19937 rng(7);
    for (int round = 0; round < 200; ++round) {
        const int N = int(rng() % 6), R = 1 + int(rng() % 3);
        const bool apart = rng() % 2, typed = rng() % 2;
        std::vector<int64_t> numel;
        std::vector<int32_t> in, out;
        for (int i = 0; i < N; ++i) {
            static const int64_t some[] = {0, 1, 2, 63, 64, 8191, 8192, 8193, 70000};
            numel.push_back(some[rng() % 9]);
            in.push_back(int32_t(rng() % 3));
            out.push_back(int32_t(rng() % 3));
        }
        std::vector<const void *> src;
        std::vector<void *> dst;
        uintptr_t next = uintptr_t(1) << 40;
        for (int r = 0; r < R; ++r)
            for (int i = 0; i < N; ++i) {
                const uintptr_t a = next + 4 * (rng() % 70);
                src.push_back(reinterpret_cast<const void *>(a));
                dst.push_back(reinterpret_cast<void *>(a + 500000 + 4 * (rng() % 70)));
                next += 1 << 20;
            }
        ddp_grads_desc d{};
        d.n_tensors = N;
        d.n_copies = R;
        d.numel = numel.data();
        d.dtype = typed ? in.data() : nullptr;
        d.grads = src.data();
        d.out = apart ? dst.data() : nullptr;
        d.out_dtype = apart && typed ? out.data() : nullptr;
        const size_t bytes = ddp_grads_workspace_bytes(&d);
        Space ws(bytes);
        d.workspace = ws.at;
        d.workspace_bytes = bytes;
        ddp_grads *g = nullptr;
        const std::string name = "list " + std::to_string(round);
        expect(ddp_grads_create(&d, &g) == DDP_OK && g, name + ": " + ddp_last_error());
        if (!g) continue;
        size_t scratch = 0;
        expect(ddp_grads_scratch_bytes(g, &scratch) == DDP_OK && scratch >= 8 && scratch <= 16384, name + ": scratch");
        Space sc(scratch);
        float norm = 0.0f;
        g_stream_device = 0;
        const hipStream_t s = reinterpret_cast<hipStream_t>(uintptr_t(0x1000));
        expect(ddp_clip_grad_norm(g, DDP_NORM_L2, 1.0f, &norm, sc.at, scratch, s) == DDP_OK, name + ": clip");
        check_tables(d, ws.at, bytes, name);
        const bool small = g_tables.all_tiles <= ddp::kSmallClip;
        auto l = launches();
        expect(l == (small ? std::vector<std::string>{"small clip"} : std::vector<std::string>{"partials", "clip"}),
               name + ": clip launches");
        if (!small) expect(size_t(g_blocks) * 8 <= scratch, name + ": partials past the scratch");
        expect(ddp_grad_norm(g, DDP_NORM_INF, &norm, sc.at, scratch, s) == DDP_OK, name + ": norm");
        l = launches();
        expect(l.size() == (g_tables.norm_tiles <= ddp::kSmallNorm ? 1u : 2u), name + ": norm launches");
        expect(ddp_clip_grads(g, 1.0f, &norm, s) == DDP_OK, name + ": given");
        l = launches();
        expect(l.size() == (g_tables.all_tiles ? 1u : 0u), name + ": given launches");
        // refusals launch nothing
        expect(ddp_grad_norm(g, 5, &norm, sc.at, scratch, s) == DDP_ERR_INVALID, name + ": unknown norm");
        expect(ddp_grad_norm(g, 2, nullptr, sc.at, scratch, s) == DDP_ERR_INVALID, name + ": no norm");
        expect(ddp_grad_norm(g, 2, &norm, nullptr, scratch, s) == DDP_ERR_INVALID, name + ": no scratch");
        expect(ddp_grad_norm(g, 2, &norm, sc.at, scratch - 1, s) == DDP_ERR_INVALID, name + ": short scratch");
        float *inside = reinterpret_cast<float *>(sc.at), *last = inside + scratch / 4 - 1;
        for (float *bad : {inside, last}) {
            expect(ddp_grad_norm(g, 2, bad, sc.at, scratch, s) == DDP_ERR_INVALID, name + ": norm in the scratch");
            expect(ddp_clip_grad_norm(g, 2, 1.0f, bad, sc.at, scratch, s) == DDP_ERR_INVALID,
                   name + ": norm in the scratch");
        }
        for (float bad : {-1.0f, __builtin_inff(), __builtin_nanf("")}) {
            expect(ddp_clip_grad_norm(g, 2, bad, &norm, sc.at, scratch, s) == DDP_ERR_INVALID, name + ": bound");
            expect(ddp_clip_grads(g, bad, &norm, s) == DDP_ERR_INVALID, name + ": bound");
        }
        for (hipStream_t special : {hipStream_t(nullptr), hipStreamLegacy, hipStreamPerThread})
            expect(ddp_grad_norm(g, 2, &norm, sc.at, scratch, special) == DDP_OK, name + ": special stream");
        launches();
        g_stream_device = 1;
        expect(ddp_grad_norm(g, 2, &norm, sc.at, scratch, s) == DDP_ERR_INVALID, name + ": other device");
        expect(ddp_clip_grad_norm(g, 2, 1.0f, &norm, sc.at, scratch, s) == DDP_ERR_INVALID, name + ": other device");
        expect(ddp_clip_grads(g, 1.0f, &norm, s) == DDP_ERR_INVALID, name + ": other device");
        expect(launches().empty(), name + ": a refused call launched");
        ddp_grads_destroy(g);
    }
}

void reducers()
{
    for (int collective : {DDP_ALL_REDUCE, DDP_REDUCE_SCATTER}) {
        for (int W : {1, 3, 8}) {
            const std::vector<int64_t> numel = {5, 20000, 1, 0, 7};
            const std::vector<int32_t> bucket = {0, 0, 1, 1, 2};
            const std::vector<int64_t> offset = {0, 20, 0, 4, 0};
            const std::vector<int64_t> sizes = {20005, 1, 7}, starts = {0, 20005, 20006};
            std::vector<std::vector<float>> flats(W, std::vector<float>(20013));
            std::vector<std::vector<float>> grads(W, std::vector<float>(20033));
            std::vector<float *> flat;
            std::vector<const void *> ptrs;
            for (int w = 0; w < W; ++w) {
                flat.push_back(flats[w].data());
                for (size_t p = 0; p < numel.size(); ++p) ptrs.push_back(grads[w].data());
            }
            ddp_reducer_desc d{};
            d.world = W;
            d.n_params = 5;
            d.param_numel = numel.data();
            d.bucket_of = bucket.data();
            d.offset_in_bucket = offset.data();
            d.n_buckets = 3;
            d.input_mode = DDP_IN_F32_COPY;
            d.grads = ptrs.data();
            d.flat = flat.data();
            d.collective = collective;
            const size_t bytes = ddp_workspace_bytes(&d);
            Space ws(bytes);
            d.workspace = ws.at;
            d.workspace_bytes = bytes;
            ddp_reducer *r = nullptr;
            const std::string name = "reducer W=" + std::to_string(W) + " collective=" + std::to_string(collective);
            expect(ddp_reducer_create(&d, &r) == DDP_OK, name + ": " + ddp_last_error());
            const size_t need = ddp_reducer_grads_workspace_bytes(r);
            expect(need > 0, name + ": size");
            Space lw(need);
            ddp_grads *g = nullptr;
            expect(ddp_grads_from_reducer(r, lw.at, need - 1, &g) == DDP_ERR_INVALID && !g, name + ": short workspace");
            expect(ddp_grads_from_reducer(r, lw.at, need, &g) == DDP_OK && g, name + ": " + ddp_last_error());
            ddp_reducer_destroy(r);   // the list keeps what it needs
            if (!g) continue;
            // what it has to hold
            std::vector<int64_t> n;
            std::vector<const void *> p;
            ddp_grads_desc want{};
            want.n_copies = 1;
            if (collective == DDP_REDUCE_SCATTER) {
                for (int b = 0; b < 3; ++b)
                    for (int c = 0; c < W; ++c) {
                        const int64_t q = (sizes[b] + W - 1) / W;
                        const int64_t lo = std::min(sizes[b], c * q), hi = std::min(sizes[b], (c + 1) * q);
                        if (lo < hi) {
                            n.push_back(hi - lo);
                            p.push_back(flat[c] + starts[b] + lo);
                        }
                    }
            } else {
                n.push_back(20013);
                for (int w = 0; w < W; ++w) p.push_back(flat[w]);
                want.n_copies = W;
            }
            want.n_tensors = int32_t(n.size());
            want.numel = n.data();
            want.grads = p.data();
            float norm;
            Space sc(16384);
            g_stream_device = 0;
            expect(ddp_clip_grad_norm(g, DDP_NORM_L2, 1.0f, &norm, sc.at, 16384, nullptr) == DDP_OK, name + ": clip");
            check_tables(want, lw.at, need, name);
            launches();
            ddp_grads_destroy(g);
        }
    }
}

void embeddings()
{
    std::mt19937 rng(11);
    int small_calls = 0, large_calls = 0;
    for (int round = 0; round < 300; ++round) {
        ddp_embedding_desc d{};
        d.n_rows = 1 + int64_t(rng() % (round % 3 ? 3000 : 900000));
        d.width = 1 + int64_t(rng() % 5000);
        d.table_stride = d.grad_stride = d.act_stride = d.width;
        d.scale = 1.0f;
        d.first_row = int64_t(rng() % 2) * 1000;
        d.padding_idx = int64_t(rng() % 3000) - 1;
        if (d.padding_idx < d.first_row || d.padding_idx >= d.first_row + d.n_rows) d.padding_idx = -1;
        d.index_dtype = DDP_I64;
        d.act_dtype = int32_t(rng() % 3);
        d.grad_dtype = int32_t(rng() % 3);
        const int64_t n = 1 + int64_t(rng() % (round % 2 ? 100 : 60000));
        const std::string name = "embedding " + std::to_string(round);
        const size_t bytes = ddp_embedding_grad_workspace_bytes(&d, n + int64_t(rng() % 5000));
        uint8_t *ws = reinterpret_cast<uint8_t *>(uintptr_t(1) << 40);
        void *p = reinterpret_cast<void *>(uintptr_t(1) << 50);
        g_stream_device = 0;
        expect(ddp_embedding_grad(&d, p, p, n, p, 1, ws, bytes, nullptr) == DDP_OK, name + ": " + ddp_last_error());
        const ddp::EmbeddingWork &w = g_work;
        const auto l = launches();
        const int vec = ddp::sum_vector(d.act_dtype, d.grad_dtype);
        if (l == std::vector<std::string>{"small grad"}) {
            const ddp::SmallPlan &q = g_small;
            expect(n <= ddp::kSmallTokens && d.width >= vec, name + ": small path taken for a large call");
            expect(q.rows >= 1 && q.rows <= ddp::kSmallRows, name + ": rows of a small range");
            expect(int64_t(q.slabs) * 64 * vec >= d.width && int64_t(q.slabs - 1) * 64 * vec < d.width,
                   name + ": slabs of the small path");
            const int64_t lds = 4 * (17 * int64_t(q.rows) + 1 + n + 16 * 64 * vec);
            expect(lds + 1024 <= 160 * 1024, name + ": LDS of the small path");
            expect(q.pad_row == -1 || q.pad_row == d.padding_idx - d.first_row, name + ": padding row");
            ++small_calls;
            continue;
        }
        ++large_calls;
        std::vector<std::string> want = {"sort", "sum"};
        if (n > w.chunk) want.push_back("join");
        expect(l == want, name + ": launches");
        expect(w.chunk >= 8 && w.chunk <= ddp::kMaxChunk && int64_t(w.n_chunks) * w.chunk >= n &&
                   int64_t(w.n_chunks - 1) * w.chunk < n,
               name + ": chunks");
        expect(w.sort_rows >= 1 && w.sort_rows <= ddp::kMaxSortRows, name + ": rows of a sorting workgroup");
        expect(w.pitch >= d.width && w.pitch % 4 == 0, name + ": pitch");
        struct Part {
            const void *at;
            size_t bytes;
        };
        const size_t slots = size_t(w.n_chunks) * size_t(w.pitch) * 4;
        const std::vector<Part> parts = {{w.row, size_t(n) * 4},
                                         {w.pos, size_t(n) * 4},
                                         {w.begin, size_t(d.n_rows + 1) * 4},
                                         {w.first, slots},
                                         {w.more, slots}};
        const uint8_t *at = ws;
        for (const Part &q : parts) {
            expect(static_cast<const uint8_t *>(q.at) >= at, name + ": parts overlap");
            expect(reinterpret_cast<uintptr_t>(q.at) % 256 == 0, name + ": a part is misaligned");
            at = static_cast<const uint8_t *>(q.at) + q.bytes;
        }
        expect(at <= ws + bytes, name + ": past the workspace");
        const hipStream_t s = reinterpret_cast<hipStream_t>(uintptr_t(0x1000));
        for (hipStream_t special : {hipStream_t(nullptr), hipStreamLegacy, hipStreamPerThread})
            expect(ddp_embedding_lookup(&d, p, p, n, p, special) == DDP_OK, name + ": special stream");
        launches();
        g_stream_device = 1;
        expect(ddp_embedding_grad(&d, p, p, n, p, 1, ws, bytes, s) == DDP_ERR_INVALID, name + ": other device");
        expect(ddp_embedding_lookup(&d, p, p, n, p, s) == DDP_ERR_INVALID, name + ": other device");
        expect(launches().empty(), name + ": a refused call launched");
    }
    expect(small_calls >= 20 && large_calls >= 20, "embeddings: one path hardly taken");
}

void exhaustion()
{
    std::vector<int64_t> numel = {10, 20000, 3};
    std::vector<const void *> src;
    for (uintptr_t i = 1; i <= 3; ++i) src.push_back(reinterpret_cast<const void *>(i << 30));
    ddp_grads_desc d{};
    d.n_tensors = 3;
    d.n_copies = 1;
    d.numel = numel.data();
    d.grads = src.data();
    const size_t bytes = ddp_grads_workspace_bytes(&d);
    Space ws(bytes);
    d.workspace = ws.at;
    d.workspace_bytes = bytes;
    bool made = false;
    fake::g_logging = false;
    for (long budget = 0; budget < 64 && !made; ++budget) {
        ddp_grads *g = nullptr;
        g_new_budget = budget;
        const int rc = ddp_grads_create(&d, &g);
        g_new_budget = -1;
        expect(rc == DDP_OK || rc == DDP_ERR_NOMEM, "exhaustion: code");
        expect((rc == DDP_OK) == (g != nullptr), "exhaustion: handle");
        made = g != nullptr;
        ddp_grads_destroy(g);
        // a refusal whose text cannot be stored is still a refusal
        g_new_budget = 0;
        expect(ddp_grad_norm(nullptr, 0, nullptr, nullptr, 0, nullptr) == DDP_ERR_INVALID, "exhaustion: refusal");
        expect(ddp_embedding_lookup(nullptr, nullptr, nullptr, 0, nullptr, nullptr) == DDP_ERR_INVALID,
               "exhaustion: refusal");
        g_new_budget = -1;
    }
    fake::g_logging = true;
    expect(made, "exhaustion: never created");
}

}  // namespace

int main()
{
    lists();
    reducers();
    embeddings();
    exhaustion();
    if (g_bad) {
        std::fprintf(stderr, "%d checks failed\n", g_bad);
        return 1;
    }
    std::printf("list_host_checks ok\n");
    return 0;
}
