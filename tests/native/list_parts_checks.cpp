// Lists around the size from which clipping into other buffers is a workgroup
// a part of a tile: which launches the calls make, that the tables cover every
// element of every copy, and that the scratch holds a partial a workgroup of
// the norm's pass and no more than kMaxPartials of them. Against stand-ins for
// the HIP runtime (fake_hip.cpp) and the kernel launchers.
#include "ddp.h"
#include "fake_hip.h"
#include "grad_list.h"

#include <algorithm>
#include <cstdio>
#include <string>
#include <vector>

#include "failing_new.h"

namespace {

int g_bad = 0;
std::vector<std::string> g_launches;
ddp::GradTables g_tables;
int g_blocks = 0;

void expect(bool ok, const std::string &what)
{
    if (!ok && g_bad++ < 30) std::fprintf(stderr, "FAILED: %s (%s)\n", what.c_str(), ddp_last_error());
}

hipError_t note(const char *what, const ddp::GradTables &t)
{
    g_launches.push_back(what);
    g_tables = t;
    return hipSuccess;
}

}  // namespace

extern "C" hipError_t hipStreamGetDevice(hipStream_t, hipDevice_t *device)
{
    *device = 0;
    return hipSuccess;
}

namespace ddp {

hipError_t launch_norm_partials(int, const GradTables &t, int blocks, void *, hipStream_t)
{
    g_blocks = blocks;
    return note("partials", t);
}
hipError_t launch_norm_finish(int, int blocks, const void *, float *, hipStream_t)
{
    expect(blocks == g_blocks, "the norm is finished over other partials");
    return note("finish", g_tables);
}
hipError_t launch_clip(int, const GradTables &t, int, const ClipFactor &f, int n, const void *, float *, hipStream_t)
{
    expect(f.norm || n == g_blocks, "the norm is taken over other partials");
    return note(f.norm ? "clip given" : "clip", t);
}
hipError_t launch_clip_parts(const GradTables &t, const ClipFactor &f, hipStream_t)
{
    expect(f.norm != nullptr, "clip parts without a norm");
    return note("parts", t);
}
hipError_t launch_small(int, const GradTables &t, bool clip, float, float *, hipStream_t)
{
    return note(clip ? "small clip" : "small", t);
}

}  // namespace ddp

namespace {

using Names = std::vector<std::string>;

Names launches()
{
    Names v;
    v.swap(g_launches);
    return v;
}

void check(const std::string &name, const std::vector<int64_t> &numel, int copies, bool apart)
{
    std::vector<const void *> src;
    std::vector<void *> dst;
    for (int r = 0; r < copies; ++r)
        for (size_t i = 0; i < numel.size(); ++i) {
            src.push_back(reinterpret_cast<const void *>((uintptr_t(1) << 40) + (src.size() << 34) + 4 * i));
            dst.push_back(reinterpret_cast<void *>((uintptr_t(1) << 46) + (dst.size() << 34) + 12 * i));
        }
    ddp_grads_desc d{};
    d.n_tensors = int32_t(numel.size());
    d.n_copies = copies;
    d.numel = numel.data();
    d.grads = src.data();
    d.out = apart ? dst.data() : nullptr;
    std::vector<uint64_t> ws(ddp_grads_workspace_bytes(&d) / 8 + 2);
    const uintptr_t at = (reinterpret_cast<uintptr_t>(ws.data()) + 15) / 16 * 16;
    d.workspace = reinterpret_cast<void *>(at);
    d.workspace_bytes = ddp_grads_workspace_bytes(&d);
    ddp_grads *g = nullptr;
    expect(ddp_grads_create(&d, &g) == DDP_OK && g, name + ": create");
    if (!g) return;
    size_t bytes = 0;
    expect(ddp_grads_scratch_bytes(g, &bytes) == DDP_OK, name + ": scratch");
    expect(bytes >= 8 && bytes <= sizeof(double) * ddp::kMaxPartials, name + ": scratch of more than 8 KiB");
    std::vector<double> scratch(bytes / 8);
    float norm = 0.0f;
    expect(ddp_clip_grad_norm(g, DDP_NORM_L2, 1.0f, &norm, scratch.data(), bytes, nullptr) == DDP_OK, name + ": clip");
    const int tiles = g_tables.all_tiles;
    const bool parts = apart && tiles > ddp::kManyTiles;
    expect(launches() == (tiles <= ddp::kSmallClip ? Names{"small clip"}
                          : parts                  ? Names{"partials", "finish", "parts"}
                                                   : Names{"partials", "clip"}),
           name + ": launches");
    if (tiles > ddp::kSmallClip) expect(size_t(g_blocks) * 8 == bytes, name + ": partials and scratch");
    expect(ddp_clip_grads(g, 1.0f, &norm, nullptr) == DDP_OK, name + ": given");
    expect(launches() == (parts ? Names{"parts"} : Names{"clip given"}), name + ": launches with a given norm");
    // every element of every copy once
    int tile = 0;
    for (size_t k = 0; k < src.size(); ++k) {
        const int64_t n = numel[k % numel.size()];
        int64_t done = 0;
        for (; done < n && tile < tiles; ++tile) {
            const ddp::GradSeg &s = g_tables.segs[g_tables.tile_seg[tile]];
            const int64_t base = int64_t(tile - s.tile0) * ddp::kGradTile - s.shift;
            expect(s.src == src[k] && s.dst == (apart ? dst[k] : src[k]) && s.len == n &&
                       std::max<int64_t>(base, 0) == done,
                   name + ": tile " + std::to_string(tile));
            done = std::min(n, base + ddp::kGradTile);
        }
        expect(done == n, name + ": tensor " + std::to_string(k));
        if (k + 1 == numel.size()) expect(tile == g_tables.norm_tiles, name + ": the norm's tiles");
    }
    expect(tile == tiles, name + ": tiles left over");
    ddp_grads_destroy(g);
}

}  // namespace

int main()
{
    const int64_t tile = ddp::kGradTile;
    for (bool apart : {false, true}) {
        const std::string where = apart ? " apart" : " in place";
        check("one below" + where, {ddp::kManyTiles * tile - 200}, 1, apart);
        check("the most" + where, {ddp::kManyTiles * tile}, 1, apart);
        check("one more" + where, {ddp::kManyTiles * tile + 1}, 1, apart);
        check("of copies" + where, {ddp::kManyTiles / 4 * tile, 5}, 4, apart);
        check("of many tensors" + where, std::vector<int64_t>(5000, 33), 1, apart);
        check("of odd tensors" + where, {9999 * tile + 77, 1, 0, 8191, 8193}, 3, apart);
        check("few" + where, {100}, 1, apart);
        check("some" + where, {100 * tile}, 1, apart);
    }
    if (g_bad) {
        std::fprintf(stderr, "%d checks failed\n", g_bad);
        return 1;
    }
    std::printf("list_parts_checks ok\n");
    return 0;
}
