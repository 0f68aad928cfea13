// The list of a reducer's results belongs to the reducer's device: made with
// another device current, its kernels would run where the buffers are not.
// Against stand-ins for the HIP runtime (fake_hip.cpp, with the current device
// set here: the link wraps hipGetDevice) and the kernel launchers.
#include "ddp.h"
#include "fake_hip.h"
#include "grad_list.h"

#include <cstdio>
#include <string>
#include <vector>

#include "failing_new.h"

namespace {

int g_bad = 0;
int g_device = 0;

void expect(bool ok, const std::string &what)
{
    if (!ok && g_bad++ < 30) std::fprintf(stderr, "FAILED: %s (%s)\n", what.c_str(), ddp_last_error());
}

}  // namespace

extern "C" hipError_t __wrap_hipGetDevice(int *device)
{
    *device = g_device;
    return hipSuccess;
}

extern "C" hipError_t hipStreamGetDevice(hipStream_t, hipDevice_t *device)
{
    *device = g_device;
    return hipSuccess;
}

namespace ddp {

hipError_t launch_norm_partials(int, const GradTables &, int, void *, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_finish(int, int, const void *, float *, hipStream_t) { return hipSuccess; }
hipError_t launch_clip(int, const GradTables &, int, const ClipFactor &, int, const void *, float *, hipStream_t)
{
    return hipSuccess;
}
hipError_t launch_clip_parts(const GradTables &, const ClipFactor &, hipStream_t) { return hipSuccess; }
hipError_t launch_small(int, const GradTables &, bool, float, float *, hipStream_t) { return hipSuccess; }

}  // namespace ddp

int main()
{
    for (int own : {0, 3}) {
        for (bool fixed : {false, true}) {
            if (fixed && own != 0) continue;   // the stand-in has a static table area on device 0 only
            const std::vector<int64_t> numel = {5000, 3};
            const std::vector<int32_t> bucket = {0, 0};
            const std::vector<int64_t> offset = {0, 20000};
            std::vector<std::vector<float>> flats(2, std::vector<float>(5003));
            std::vector<float *> flat = {flats[0].data(), flats[1].data()};
            ddp_reducer_desc d{};
            d.world = 2;
            d.n_params = 2;
            d.param_numel = numel.data();
            d.bucket_of = bucket.data();
            d.offset_in_bucket = offset.data();
            d.n_buckets = 1;
            d.input_mode = DDP_IN_F32_VIEW;
            d.flat = flat.data();
            std::vector<uint64_t> ws(ddp_workspace_bytes(&d) / 8 + 2);
            const std::string name = "device " + std::to_string(own) + (fixed ? " static" : "");
            g_device = own;
            ddp_reducer *r = nullptr;
            if (fixed) {
                expect(ddp_reducer_create_static(&d, &r) == DDP_OK, name + ": create");
            } else {
                d.workspace = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(ws.data()) + 15) / 16 * 16);
                d.workspace_bytes = ddp_workspace_bytes(&d);
                expect(ddp_reducer_create(&d, &r) == DDP_OK, name + ": create");
            }
            if (!r) continue;
            const size_t need = ddp_reducer_grads_workspace_bytes(r);
            std::vector<uint64_t> lw(need / 8 + 4);
            void *at = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(lw.data()) + 15) / 16 * 16);
            for (int other : {own + 1, own + 2}) {
                g_device = other;
                ddp_grads *g = nullptr;
                expect(ddp_grads_from_reducer(r, at, need, &g) == DDP_ERR_INVALID && !g, name + ": another device");
                expect(std::string(ddp_last_error()).find("the reducer is on device") == 0, name + ": message");
                ddp_grads_destroy(g);
            }
            g_device = own;
            ddp_grads *g = nullptr;
            expect(ddp_grads_from_reducer(r, at, need, &g) == DDP_OK && g, name + ": its own device");
            ddp_grads_destroy(g);
            ddp_reducer_destroy(r);
        }
    }
    if (g_bad) {
        std::fprintf(stderr, "%d checks failed\n", g_bad);
        return 1;
    }
    std::printf("list_device_checks ok\n");
    return 0;
}
