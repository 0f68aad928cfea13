// The host half of the AdamW step against stand-ins for the HIP runtime, the
// library's error recording and the kernel's launcher (below), built under
// AddressSanitizer and UndefinedBehaviorSanitizer. Checks:
//  * the uploaded tables cover every element of every tensor exactly once,
//    inside the workspace asked for: cut at parameter addresses that are
//    multiples of 256 bytes with 32-bit states, at whole blocks with 8-bit ones;
//  * a step's scalars, and which calls are refused before a launch;
//  * the powers that the device shares with the host;
//  * host memory exhaustion gives DDP_ERR_NOMEM and leaks nothing.
#include "adamw.h"
#include "ddp.h"
#include "host_common.h"

#include <cmath>
#include <cstdio>
#include <cstring>
#include <limits>
#include <random>
#include <string>
#include <vector>

#include "failing_new.h"

namespace {

int g_bad = 0, g_device = 0, g_stream_device = 0, g_launches = 0;
char g_error[512];
ddp::AdamTables g_tables;
ddp::AdamArgs g_args;

void expect(bool ok, const std::string &what)
{
    if (!ok && g_bad++ < 30) std::fprintf(stderr, "FAILED: %s (%s)\n", what.c_str(), g_error);
}

}  // namespace

extern "C" hipError_t hipGetDevice(int *d)
{
    *d = g_device;
    return hipSuccess;
}
extern "C" hipError_t hipMemcpy(void *to, const void *from, size_t n, hipMemcpyKind)
{
    std::memcpy(to, from, n);
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
hipError_t launch_adamw(const AdamTables &t, const AdamArgs &a, hipStream_t)
{
    g_tables = t;
    g_args = a;
    ++g_launches;
    return hipSuccess;
}

}  // namespace ddp

namespace {

// Memory of exactly n bytes at a multiple of 16, so that a write behind it is
// caught.
struct Space {
    std::vector<uint8_t> bytes;
    void *at;
    explicit Space(size_t n) : bytes(n + 16)
    {
        const uintptr_t p = reinterpret_cast<uintptr_t>(bytes.data());
        const size_t skip = (16 - p % 16) % 16;
        bytes.resize(n + skip);   // shrinks: the address stays
        at = bytes.data() + skip;
    }
};

void *address(uintptr_t p)
{
    return reinterpret_cast<void *>(p);
}

// A random list at made-up addresses, and its desc.
struct List {
    std::vector<int64_t> numel;
    std::vector<int32_t> grad_type, param_type, copy_type;
    std::vector<const void *> grads;
    std::vector<void *> params, copies, m, v;
    std::vector<float *> ms, vs;
    std::vector<double> decay;
    ddp_adamw_desc d{};

    List(std::mt19937 &rng, bool small)
    {
        uintptr_t at = uintptr_t(1) << 40;
        const auto take = [&](uintptr_t size, uintptr_t count) {
            at += size * (rng() % 70);
            const uintptr_t p = (at + size - 1) / size * size;
            at = p + size * count;
            return p;
        };
        const int n = int(rng() % 12);
        for (int i = 0; i < n; ++i) {
            static const int64_t sizes[] = {0, 1, 127, 128, 129, 2047, 2048, 2049, 4096, 70001};
            const int64_t k = sizes[rng() % 10];
            numel.push_back(k);
            grad_type.push_back(int32_t(rng() % 3));
            param_type.push_back(int32_t(rng() % 3));
            copy_type.push_back(int32_t(1 + rng() % 2));
            grads.push_back(address(take(grad_type.back() ? 2 : 4, uintptr_t(k))));
            params.push_back(address(take(param_type.back() ? 2 : 4, uintptr_t(k))));
            copies.push_back(param_type.back() == DDP_F32 && rng() % 2 ? address(take(2, uintptr_t(k))) : nullptr);
            m.push_back(address(take(small ? 1 : 4, uintptr_t(k))));
            v.push_back(address(take(small ? 1 : 4, uintptr_t(k))));
            ms.push_back(static_cast<float *>(address(take(4, uintptr_t(k + 127) / 128))));
            vs.push_back(static_cast<float *>(address(take(4, uintptr_t(k + 127) / 128))));
            decay.push_back(double(rng() % 3) * 0.1);
        }
        d.n_tensors = n;
        d.state = small ? DDP_STATE_8BIT : DDP_STATE_F32;
        d.numel = numel.data();
        d.grad_dtype = grad_type.data();
        d.param_dtype = param_type.data();
        d.grads = grads.data();
        d.params = params.data();
        d.copies = copies.data();
        d.copy_dtype = copy_type.data();
        d.m = m.data();
        d.v = v.data();
        d.m_scale = small ? ms.data() : nullptr;
        d.v_scale = small ? vs.data() : nullptr;
        d.weight_decay = decay.data();
    }
};

ddp_adamw_args usual()
{
    ddp_adamw_args a{};
    a.lr = 1e-3;
    a.beta1 = 0.9;
    a.beta2 = 0.999;
    a.eps = 1e-8;
    a.step = 3;
    return a;
}

void lists()
{
    std::mt19937 rng(7);
    for (int round = 0; round < 400; ++round) {
        const bool small = round % 2;
        List l(rng, small);
        const std::string name = "list " + std::to_string(round);
        const size_t bytes = ddp_adamw_workspace_bytes(&l.d);
        Space ws(bytes);
        l.d.workspace = ws.at;
        l.d.workspace_bytes = bytes;
        ddp_adamw *o = nullptr;
        expect(ddp_adamw_create(&l.d, &o) == DDP_OK && o, name + ": create");
        if (!o) continue;
        const ddp_adamw_args a = usual();
        const int before = g_launches;
        expect(ddp_adamw_step(o, &a, nullptr) == DDP_OK, name + ": step");
        int64_t total = 0;
        for (int64_t k : l.numel) total += k;
        expect(g_launches - before == (total > 0), name + ": launches");
        if (total > 0) {
            const ddp::AdamTables &t = g_tables;
            expect(t.bits == (small ? 8 : 32), name + ": bits");
            const uint8_t *lo = static_cast<const uint8_t *>(ws.at), *hi = lo + bytes;
            expect(reinterpret_cast<const uint8_t *>(t.segs) >= lo &&
                       reinterpret_cast<const uint8_t *>(t.tile_seg + t.tiles) <= hi,
                   name + ": tables outside the workspace");
            int32_t tile = 0;
            const ddp::AdamSeg *s = t.segs;
            for (size_t i = 0; i < l.numel.size(); ++i) {
                if (l.numel[i] == 0) continue;
                const int size = l.param_type[i] ? 2 : 4;
                expect(s->grad == l.grads[i] && s->param == l.params[i] && s->copy == l.copies[i] && s->m == l.m[i] &&
                           s->v == l.v[i] && s->len == l.numel[i] && s->decay == l.decay[i] && s->tile0 == tile &&
                           s->type == l.grad_type[i],
                       name + ": record");
                const uintptr_t cut = reinterpret_cast<uintptr_t>(s->param) - uintptr_t(s->shift * size);
                expect(small ? s->shift == 0 && s->m_scale == l.ms[i] && s->v_scale == l.vs[i] : cut % 256 == 0,
                       name + ": cut");
                // the tensor's tiles cover [-shift, ...) without a gap, and no more than needed
                int64_t covered = -int64_t(s->shift);
                for (; tile < t.tiles && t.tile_seg[tile] == s - t.segs; ++tile) {
                    expect(covered < s->len, name + ": a tile past the tensor");
                    covered += ddp::kAdamTile;
                }
                expect(covered >= s->len, name + ": elements without a tile");
                ++s;
            }
            expect(tile == t.tiles, name + ": tiles without a tensor");
        }
        ddp_adamw_destroy(o);
    }
}

void steps()
{
    std::mt19937 rng(3);
    int64_t numel = 5000;
    const void *grad = address(uintptr_t(1) << 40);
    void *param = address(uintptr_t(2) << 40), *m = address(uintptr_t(3) << 40), *v = address(uintptr_t(4) << 40);
    ddp_adamw_desc d{};
    d.n_tensors = 1;
    d.numel = &numel;
    d.grads = &grad;
    d.params = &param;
    d.m = &m;
    d.v = &v;
    const size_t bytes = ddp_adamw_workspace_bytes(&d);
    Space ws(bytes);
    d.workspace = ws.at;
    d.workspace_bytes = bytes;
    ddp_adamw *o = nullptr;
    expect(ddp_adamw_create(&d, &o) == DDP_OK, "steps: create");
    if (!o) return;
    const float *norm = static_cast<const float *>(address(uintptr_t(5) << 40));
    const double inf = std::numeric_limits<double>::infinity(), nan = std::nan("");
    const auto refused = [&](const char *what, ddp_adamw_args a) {
        const int before = g_launches;
        expect(ddp_adamw_step(o, &a, nullptr) == DDP_ERR_INVALID && g_launches == before, std::string("refusal of ") + what);
    };
    const auto taken = [&](const char *what, ddp_adamw_args a) {
        const int before = g_launches;
        expect(ddp_adamw_step(o, &a, nullptr) == DDP_OK && g_launches == before + 1, what);
    };
    ddp_adamw_args a;
    for (double bad : {-1e-3, inf, nan}) {
        a = usual(), a.lr = bad, refused("lr", a);
        a = usual(), a.eps = bad, refused("eps", a);
    }
    for (double bad : {1e-39, 1e-50, 1e39, -1e-50}) a = usual(), a.eps = bad, refused("eps beyond fp32's normal numbers", a);
    for (double good : {0.0, 1e-37, 1e-8, 1.0}) a = usual(), a.eps = good, taken("eps", a);
    for (double bad : {-0.1, 1.0, 1.5, inf, nan}) {
        a = usual(), a.beta1 = bad, refused("beta1", a);
        a = usual(), a.beta2 = bad, refused("beta2", a);
    }
    for (int64_t bad : {int64_t(0), int64_t(-1), std::numeric_limits<int64_t>::min()}) a = usual(), a.step = bad, refused("step", a);
    a = usual(), a.norm = norm, a.max_norm = -1.0f, refused("max_norm", a);
    a = usual(), a.norm = norm, a.max_norm = float(nan), refused("max_norm", a);
    a = usual(), a.skip_nonfinite = 1, refused("skip without a norm", a);
    a = usual(), a.norm = reinterpret_cast<const float *>(uintptr_t(norm) + 2), refused("a misaligned norm", a);
    a = usual(), a.step_ptr = reinterpret_cast<const int64_t *>(uintptr_t(norm) + 4), refused("a misaligned step", a);
    for (void *p : {param, m, v}) {
        const uintptr_t last = uintptr_t(p) + 4 * 4999;
        a = usual(), a.norm = reinterpret_cast<const float *>(last), refused("a norm among what is written", a);
        a = usual(), a.lr_ptr = reinterpret_cast<const float *>(last), refused("a rate among what is written", a);
        a = usual(), a.step_ptr = reinterpret_cast<const int64_t *>(uintptr_t(p) + 4 * 4992), refused("a step among what is written", a);
        a = usual(), a.norm = reinterpret_cast<const float *>(last + 4), taken("a norm behind a tensor", a);
    }
    a = usual(), a.norm = static_cast<const float *>(grad), taken("a norm among the gradients, which are read only", a);
    a = usual(), a.lr = nan, a.lr_ptr = norm, taken("a rate on the device", a);
    a = usual(), a.step = 0, a.step_ptr = reinterpret_cast<const int64_t *>(norm), taken("a step on the device", a);
    a = usual(), a.norm = norm, a.max_norm = float(inf), taken("no bound", a);
    for (int64_t t : {int64_t(1), int64_t(2), int64_t(3), int64_t(1000), int64_t(1) << 62}) {
        a = usual(), a.step = t, taken("step", a);
        const double b1 = std::pow(a.beta1, double(t)), b2 = std::pow(a.beta2, double(t));
        expect(std::fabs(g_args.size / (a.lr / (1.0 - b1)) - 1.0) < 1e-7, "size");
        expect(std::fabs(g_args.root * std::sqrt(1.0 - b2) - 1.0) < 1e-7, "root");
        expect(g_args.b1 == 0.9f && g_args.a1 == float(1.0 - 0.9) && g_args.b2 == 0.999f && g_args.a2 == float(1.0 - 0.999),
               "rates");
    }
    a = usual();
    g_stream_device = 1;
    expect(ddp_adamw_step(o, &a, static_cast<hipStream_t>(address(0x1000))) == DDP_ERR_INVALID, "stream of another device");
    g_stream_device = 0;
    g_device = 1;
    expect(ddp_adamw_step(o, &a, nullptr) == DDP_ERR_INVALID, "another device");
    g_device = 0;
    expect(ddp_adamw_step(o, nullptr, nullptr) == DDP_ERR_INVALID, "no args");
    ddp_adamw_destroy(o);
}

void powers()
{
    expect(ddp::power(0.5, 0) == 1.0 && ddp::power(0.0, 0) == 1.0 && ddp::power(0.0, 5) == 0.0, "power: ends");
    for (double b : {0.1, 0.9, 0.95, 0.999, 0.9999})
        for (int64_t t : {1, 2, 3, 10, 999, 12345}) {
            const double want = std::pow(b, double(t)), got = ddp::power(b, t);
            expect(want < 0x1p-60 ? got == 0.0 : std::fabs(got - want) <= want * double(t + 2) * 2.3e-16, "power");
            expect(std::fabs((1.0 - got) - (1.0 - want)) <= 1e-13, "power: distance from 1");
        }
    expect(ddp::power(0.999, std::numeric_limits<int64_t>::max()) == 0.0, "power: vanishes");
}

void exhaustion()
{
    std::mt19937 rng(5);
    List l(rng, true);
    while (l.numel.size() < 4) l = List(rng, true);
    const size_t bytes = ddp_adamw_workspace_bytes(&l.d);
    Space ws(bytes);
    l.d.workspace = ws.at;
    l.d.workspace_bytes = bytes;
    bool made = false;
    for (long budget = 0; budget < 64 && !made; ++budget) {
        ddp_adamw *o = nullptr;
        g_new_budget = budget;
        const int rc = ddp_adamw_create(&l.d, &o);
        g_new_budget = -1;
        expect(rc == DDP_OK || rc == DDP_ERR_NOMEM, "exhaustion: code");
        expect((rc == DDP_OK) == (o != nullptr), "exhaustion: handle");
        made = o != nullptr;
        ddp_adamw_destroy(o);
    }
    expect(made, "exhaustion: never created");
}

}  // namespace

int main()
{
    lists();
    steps();
    powers();
    exhaustion();
    if (g_bad) {
        std::fprintf(stderr, "%d checks failed\n", g_bad);
        return 1;
    }
    std::printf("adamw_host_checks ok\n");
    return 0;
}
