// Calls on gradient lists that would write over what they read, against
// stand-ins for the HIP runtime (fake_hip.cpp) and the kernel launchers
// (below), built under AddressSanitizer and UndefinedBehaviorSanitizer: a norm
// or a scratch at every kind of place around a list's tensors, their other
// buffers and its tables. A refused call launches nothing.
#include "ddp.h"
#include "embedding.h"
#include "fake_hip.h"
#include "grad_list.h"

#include <cstdio>
#include <string>
#include <vector>

#include "failing_new.h"

namespace {

int g_bad = 0;
int g_launches = 0;

void expect(bool ok, const std::string &what)
{
    if (!ok && g_bad++ < 30) std::fprintf(stderr, "FAILED: %s\n", what.c_str());
}

hipError_t launched()
{
    ++g_launches;
    return hipSuccess;
}

}  // namespace

extern "C" hipError_t hipStreamGetDevice(hipStream_t, hipDevice_t *device)
{
    *device = 0;
    return hipSuccess;
}

namespace ddp {

hipError_t launch_norm_partials(int, const GradTables &, int, void *, hipStream_t) { return launched(); }
hipError_t launch_norm_finish(int, int, const void *, float *, hipStream_t) { return launched(); }
hipError_t launch_clip(int, const GradTables &, int, const ClipFactor &, int, const void *, float *, hipStream_t)
{
    return launched();
}
hipError_t launch_clip_parts(const GradTables &, const ClipFactor &, hipStream_t) { return launched(); }
hipError_t launch_small(int, const GradTables &, bool, float, float *, hipStream_t) { return launched(); }

}  // namespace ddp

namespace {

struct List {
    ddp_grads *g = nullptr;
    std::vector<uint8_t> store;
    uintptr_t ws = 0;
    size_t ws_bytes = 0, scratch_bytes = 0;

    List(const std::vector<int64_t> &numel, int copies, const std::vector<uintptr_t> &src,
         const std::vector<uintptr_t> &dst)
    {
        ddp_grads_desc d{};
        d.n_tensors = int32_t(numel.size());
        d.n_copies = copies;
        d.numel = numel.data();
        d.grads = reinterpret_cast<const void *const *>(src.data());
        d.out = dst.empty() ? nullptr : reinterpret_cast<void *const *>(dst.data());
        ws_bytes = ddp_grads_workspace_bytes(&d);
        store.resize(ws_bytes + 256);
        ws = (reinterpret_cast<uintptr_t>(store.data()) + 255) / 256 * 256;
        d.workspace = reinterpret_cast<void *>(ws);
        d.workspace_bytes = ws_bytes;
        expect(ddp_grads_create(&d, &g) == DDP_OK && g, std::string("create: ") + ddp_last_error());
        expect(ddp_grads_scratch_bytes(g, &scratch_bytes) == DDP_OK, "scratch");
    }
    ~List() { ddp_grads_destroy(g); }

    // What the three calls give for a norm and a scratch at these addresses.
    void calls(uintptr_t norm, uintptr_t scratch, bool norm_ok, bool clip_ok, const std::string &name) const
    {
        float *n = reinterpret_cast<float *>(norm);
        void *s = reinterpret_cast<void *>(scratch);
        g_launches = 0;
        expect((ddp_grad_norm(g, 2, n, s, scratch_bytes, nullptr) == DDP_OK) == norm_ok, name + ": the norm");
        expect((g_launches > 0) == norm_ok, name + ": the norm's launches");
        g_launches = 0;
        expect((ddp_clip_grad_norm(g, 2, 1.0f, n, s, scratch_bytes, nullptr) == DDP_OK) == clip_ok, name + ": clipping");
        expect((g_launches > 0) == clip_ok, name + ": clipping's launches");
    }
    void given(uintptr_t norm, bool ok, const std::string &name) const
    {
        g_launches = 0;
        const int rc = ddp_clip_grads(g, 1.0f, reinterpret_cast<const float *>(norm), nullptr);
        expect((rc == DDP_OK) == ok && (g_launches > 0) == ok, name + ": a given norm");
    }
};

constexpr uintptr_t kFree = uintptr_t(1) << 45;   // nothing lies there

void check(const std::string &name, const std::vector<int64_t> &numel, int copies, bool apart)
{
    std::vector<uintptr_t> src, dst;
    for (int r = 0; r < copies; ++r)
        for (size_t i = 0; i < numel.size(); ++i) {
            src.push_back((uintptr_t(1) << 40) + (src.size() << 32) + 4 * i);
            if (apart) dst.push_back((uintptr_t(1) << 42) + (dst.size() << 32) + 8 * i);
        }
    const List l(numel, copies, src, dst);
    l.calls(kFree, kFree + 64, true, true, name + " apart");
    l.given(kFree, true, name + " apart");
    const uintptr_t sc = l.scratch_bytes;
    for (size_t k = 0; k < src.size(); ++k) {
        const uintptr_t bytes = 4 * uintptr_t(numel[k % numel.size()]);
        if (!bytes) continue;
        const std::string t = name + " tensor " + std::to_string(k);
        const uintptr_t a = src[k], even = a + 8 - a % 8;   // a scratch lies at multiples of 8
        for (uintptr_t in : {a, a + bytes - 4, a + bytes / 8 * 4}) {
            l.calls(in, kFree, false, false, t + ": norm inside");
            l.given(in, apart, t + ": norm inside");
        }
        l.calls(a - 4, kFree, true, true, t + ": norm right before");
        l.calls(a + bytes, kFree, true, true, t + ": norm right behind");
        l.given(a - 4, true, t + ": norm right before");
        l.given(a + bytes, true, t + ": norm right behind");
        l.calls(kFree, even - 8, false, false, t + ": scratch at its beginning");
        l.calls(kFree, (a + bytes - 1) / 8 * 8, false, false, t + ": scratch at its end");
        l.calls(kFree, a / 8 * 8 - sc, true, true, t + ": scratch right before");
        l.calls(kFree, (a + bytes + 7) / 8 * 8, true, true, t + ": scratch right behind");
        if (!apart) continue;
        const uintptr_t o = dst[k];
        for (uintptr_t in : {o, o + bytes - 4}) {
            l.calls(in, kFree, true, false, t + ": norm in its other buffer");
            l.given(in, false, t + ": norm in its other buffer");
        }
        l.calls(kFree, o / 8 * 8, true, false, t + ": scratch in its other buffer");
        l.calls(o + bytes, kFree, true, true, t + ": norm behind its other buffer");
    }
    for (uintptr_t in : {l.ws, l.ws + l.ws_bytes - 4}) l.calls(in, kFree, false, false, name + ": norm in the tables");
    l.calls(kFree, l.ws, false, false, name + ": scratch in the tables");
    l.calls(kFree, l.ws - sc + 8, false, false, name + ": scratch that reaches the tables");
    l.calls(kFree, l.ws + l.ws_bytes, true, true, name + ": scratch behind the tables");
}

// Tensors side by side are one stretch: the border between two is inside.
void side_by_side()
{
    const uintptr_t a = uintptr_t(1) << 40;
    const List l({100, 50, 7}, 1, {a + 200, a, a + 600}, {});   // [a, a + 628)
    for (uintptr_t in : {a + 196, a + 200, a + 596, a + 600, a + 624}) l.calls(in, kFree, false, false, "side by side");
    l.calls(a + 628, kFree, true, true, "behind the last");
    l.calls(a - 4, kFree, true, true, "before the first");
}

}  // namespace

int main()
{
    for (bool apart : {false, true}) {
        const std::string where = apart ? " apart" : " in place";
        check("few" + where, {5, 0, 900, 1}, 1, apart);
        check("copies" + where, {700, 33}, 4, apart);
        check("tiles" + where, {9 * ddp::kGradTile + 1, 20000}, 2, apart);
        check("many tiles" + where, {int64_t(ddp::kManyTiles + 9) * ddp::kGradTile}, 1, apart);
    }
    side_by_side();
    const List none({}, 1, {}, {});
    float norm = 0.0f;
    none.calls(reinterpret_cast<uintptr_t>(&norm), kFree, true, true, "empty");
    if (g_bad) {
        std::fprintf(stderr, "%d checks failed\n", g_bad);
        return 1;
    }
    std::printf("list_alias_checks ok\n");
    return 0;
}
