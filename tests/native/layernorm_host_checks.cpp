// The host half of the layer norm against stand-ins for the HIP runtime, the
// library's error recording and the kernels' launchers (below), built under
// AddressSanitizer and UndefinedBehaviorSanitizer. Checks:
//  * which overlaps of strided arguments are refused, against every byte's
//    owner: none that meets passes, and none of one stride that does not is
//    refused;
//  * that the parts of a gradient call fit the workspace, and which launches it
//    makes;
//  * another device, special streams, and host memory exhaustion.
#include "ddp.h"
#include "host_common.h"
#include "layernorm.h"

#include <cstdio>
#include <map>
#include <random>
#include <string>
#include <vector>

#include "failing_new.h"

namespace {

int g_bad = 0, g_stream_device = 0, g_launches = 0;
std::string g_made;
char g_error[512];
ddp::LayerBackward g_back;

void expect(bool ok, const std::string &what)
{
    if (!ok && g_bad++ < 30) std::fprintf(stderr, "FAILED: %s (%s)\n", what.c_str(), g_error);
}

hipError_t note(const char *what)
{
    ++g_launches;
    g_made += what;
    return hipSuccess;
}

template <class T = void>
T *address(uintptr_t p)
{
    return reinterpret_cast<T *>(p);
}

}  // namespace

extern "C" hipError_t hipGetDevice(int *d)
{
    *d = 0;
    return hipSuccess;
}

namespace ddp {

int fail(int code, const char *msg) noexcept
{
    std::snprintf(g_error, sizeof g_error, "%s", msg);
    return code;
}
int fail(int code, const std::string &msg) noexcept { return fail(code, msg.c_str()); }
int hip_fail(const char *what, hipError_t) noexcept { return fail(DDP_ERR_HIP, what); }
int no_memory() noexcept { return fail(DDP_ERR_NOMEM, "out of memory"); }
int check_stream(hipStream_t s, int device)
{
    return !s || g_stream_device == device ? int(DDP_OK) : fail(DDP_ERR_INVALID, "stream of another device");
}
hipError_t launch_layernorm(const LayerArgs &, const LayerForward &, hipStream_t) { return note("forward "); }
hipError_t launch_layernorm_rows(const LayerArgs &, const LayerBackward &b, hipStream_t)
{
    g_back = b;
    return note("rows ");
}
hipError_t launch_layernorm_wide(const LayerArgs &, const LayerBackward &b, hipStream_t)
{
    g_back = b;
    return note("wide ");
}
hipError_t launch_layernorm_small(const LayerArgs &, const LayerBackward &b, hipStream_t)
{
    g_back = b;
    return note("small ");
}
hipError_t launch_layernorm_join(const LayerArgs &, const LayerBackward &b, hipStream_t)
{
    g_back = b;
    return note("join ");
}

}  // namespace ddp

namespace {

ddp_layernorm_desc desc_of(int64_t width)
{
    ddp_layernorm_desc d{};
    d.width = d.x_stride = d.add_stride = d.z_stride = d.y_stride = width;
    d.eps = 1e-5f;
    return d;
}

// x and y as strided rows over a small range of bytes.
void overlaps()
{
    std::mt19937 rng(11);
    int met = 0, apart = 0;
    for (int round = 0; round < 30000; ++round) {
        ddp_layernorm_desc d = desc_of(1 + int64_t(rng() % 6));
        d.x_stride += int64_t(rng() % 12);
        d.y_stride = rng() % 2 ? d.x_stride : d.width + int64_t(rng() % 12);
        d.y_dtype = rng() % 3 == 0 ? DDP_BF16 : DDP_F32;
        const int64_t n = 1 + int64_t(rng() % 5);
        const int64_t ysz = d.y_dtype == DDP_F32 ? 4 : 2;
        const uintptr_t x = 0x10000, y = x + 4 * (rng() % 80) - 160;
        std::map<uintptr_t, int> owner;
        for (int64_t r = 0; r < n; ++r)
            for (int64_t b = 0; b < 4 * d.width; ++b) owner[x + uintptr_t(4 * r * d.x_stride + b)] = 1;
        bool meet = false;
        for (int64_t r = 0; r < n; ++r)
            for (int64_t b = 0; b < ysz * d.width; ++b) meet |= owner.count(y + uintptr_t(ysz * r * d.y_stride + b)) > 0;
        const bool same = x == y && ysz == 4 && (n == 1 || d.x_stride == d.y_stride);
        const int rc = ddp_layernorm(&d, n, address(x), nullptr, nullptr, nullptr, nullptr, address(y), nullptr, nullptr,
                                     nullptr);
        const std::string name = "overlap " + std::to_string(round);
        if (same || (!meet && (n == 1 || 4 * d.x_stride == ysz * d.y_stride)))
            expect(rc == DDP_OK, name + ": refused");
        if (meet && !same) expect(rc == DDP_ERR_INVALID, name + ": passed");
        (meet ? met : apart)++;
    }
    expect(met > 1000 && apart > 1000, "overlaps: one side hardly met");
}

void gradients()
{
    std::mt19937 rng(5);
    int wide = 0, held = 0, small = 0;
    for (int round = 0; round < 3000; ++round) {
        static const int64_t widths[] = {1, 3, 8, 512, 513, 1024, 1025, 2048, 8192, 8193, 16384, 16385, 100000, 1 << 20};
        ddp_layernorm_desc d = desc_of(widths[rng() % 14]);
        d.kind = int32_t(rng() % 2);
        d.x_dtype = int32_t(rng() % 3);
        d.y_dtype = d.x_dtype ? d.x_dtype : int32_t(rng() % 3);
        const int64_t n = rng() % 4 ? 1 + int64_t(rng() % 5000) : int64_t(rng() % 3);
        const size_t bytes = ddp_layernorm_grad_workspace_bytes(&d, n + int64_t(rng() % 100));
        const uintptr_t far = uintptr_t(1) << 40;
        void *dw = rng() % 4 ? address(5 * far) : nullptr, *db = rng() % 2 ? address(6 * far) : nullptr;
        void *dx = rng() % 3 ? address(7 * far) : nullptr, *ws = address(8 * far);
        const int32_t acc = int32_t(rng() % 2);
        g_made.clear();
        const std::string name = "gradient " + std::to_string(round);
        expect(ddp_layernorm_grad(&d, n, address(far), address(2 * far), nullptr, nullptr, address<float>(3 * far),
                                  address<float>(4 * far), dx, dw, db, acc, ws, bytes, nullptr) == DDP_OK,
               name);
        const bool sums = dw || db;
        std::string want;
        const bool reads_again = d.width > 2048 * ddp::layer_vector(d.x_dtype, d.y_dtype);
        const int64_t each = (d.x_dtype ? 2 : 4) + (d.y_dtype ? 2 : 4);
        const int64_t data = n * d.width * each;
        if (sums && n > 0 && n <= 2048 && !reads_again && data <= 8 << 20 && n * data <= int64_t(1) << 33) {
            want = "small ";
            ++small;
        } else {
            if (n > 0 && (dx || sums)) want += reads_again ? "wide " : "rows ";
            if (sums && (n > 0 || !acc)) want += "join ";
        }
        expect(g_made == want, name + ": launches " + g_made);
        if (!want.empty()) {
            expect((g_back.parts != nullptr) == sums, name + ": parts");
            expect(size_t(g_back.n_parts) * 8 * size_t(d.width) <= bytes, name + ": parts outside the workspace");
            expect(n == 0 || (g_back.n_parts > 0 && g_back.n_parts <= 2048), name + ": number of parts");
            expect((g_back.mean != nullptr) == (d.kind == DDP_LAYER_NORM), name + ": mean");
            (reads_again ? wide : held)++;
        }
    }
    expect(wide > 100 && held > 100 && small > 100, "gradients: one path hardly taken");
    ddp_layernorm_desc d = desc_of(16);
    const uintptr_t far = uintptr_t(1) << 40;
    g_made.clear();   // one launch would read dy while it writes dx there
    expect(ddp_layernorm_grad(&d, 2, address(far), address(2 * far), nullptr, nullptr, address<float>(3 * far),
                              address<float>(4 * far), address(far), address(5 * far), nullptr, 0, address(6 * far), 4096,
                              nullptr) == DDP_OK && g_made == "rows join ", "gradient in dy's place: " + g_made);
    g_stream_device = 1;
    hipStream_t s = static_cast<hipStream_t>(address(0x1000));
    const int before = g_launches;
    expect(ddp_layernorm(&d, 2, address(far), nullptr, nullptr, nullptr, nullptr, address(2 * far), nullptr, nullptr, s) ==
               DDP_ERR_INVALID, "forward: stream of another device");
    expect(ddp_layernorm_grad(&d, 2, address(far), address(2 * far), nullptr, nullptr, address<float>(3 * far),
                              address<float>(4 * far), address(5 * far), nullptr, nullptr, 0, nullptr, 0, s) ==
               DDP_ERR_INVALID, "gradient: stream of another device");
    expect(g_launches == before, "a launch on another device's stream");
    g_stream_device = 0;
}

void exhaustion()
{
    const uintptr_t far = uintptr_t(1) << 40;
    ddp_layernorm_desc d = desc_of(16);
    bool made = false;
    for (long budget = 0; budget < 64 && !made; ++budget) {
        const int before = g_launches;
        g_new_budget = budget;
        const int rc = ddp_layernorm(&d, 2, address(far), address(2 * far), address(3 * far), address(4 * far),
                                     address(5 * far), address(6 * far), address<float>(7 * far), address<float>(8 * far),
                                     nullptr);
        const int rc2 = ddp_layernorm_grad(&d, 2, address(far), address(2 * far), address(3 * far), address(4 * far),
                                           address<float>(5 * far), address<float>(6 * far), address(7 * far),
                                           address(8 * far), address(9 * far), 1, address(10 * far), 1 << 20, nullptr);
        g_new_budget = -1;
        expect((rc == DDP_OK || rc == DDP_ERR_NOMEM) && (rc2 == DDP_OK || rc2 == DDP_ERR_NOMEM), "exhaustion: code");
        made = rc == DDP_OK && rc2 == DDP_OK;
        expect(made || g_launches - before < 3, "exhaustion: launches");
    }
    expect(made, "exhaustion: never launched");
}

}  // namespace

int main()
{
    overlaps();
    gradients();
    exhaustion();
    if (g_bad) {
        std::fprintf(stderr, "%d checks failed\n", g_bad);
        return 1;
    }
    std::printf("layernorm_host_checks ok\n");
    return 0;
}
