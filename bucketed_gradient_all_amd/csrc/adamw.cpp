// Host half of the AdamW step: validation, the tile tables, the scalars of a
// step and its launch.
#include "adamw.h"
#include "host_common.h"
#include "spans.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <memory>
#include <vector>

using ddp::AdamArgs;
using ddp::AdamSeg;
using ddp::AdamTables;
using ddp::fail;
using ddp::guarded;
using ddp::hip_fail;
using ddp::kAdamTile;
using ddp::kStateBlock;
using ddp::meets;
using ddp::Spans;

struct ddp_adamw {
    AdamTables tables{};
    Spans written;   // parameters, copies and states
    int device = -1;
};

namespace {

constexpr size_t kAlign = 16;

// Tiles of a list, at most: 2^40 elements.
constexpr int64_t kMostTiles = int64_t(1) << 30;

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

int32_t type_of(const int32_t *types, int32_t i)
{
    return types ? types[i] : int32_t(DDP_F32);
}

std::string tensor(int32_t i)
{
    return "tensor " + std::to_string(i);
}

// Everything of a desc but its pointers' values.
int check_sizes(const ddp_adamw_desc *d)
{
    if (!d) return fail(DDP_ERR_INVALID, "desc is NULL");
    if (d->n_tensors < 0) return fail(DDP_ERR_INVALID, "n_tensors is negative");
    if (d->state != DDP_STATE_F32 && d->state != DDP_STATE_8BIT)
        return fail(DDP_ERR_INVALID, "unknown state " + std::to_string(d->state));
    if (d->n_tensors > 0 && !d->numel) return fail(DDP_ERR_INVALID, "numel is NULL");
    if (!d->copies != !d->copy_dtype) return fail(DDP_ERR_INVALID, "copies and copy_dtype go together");
    int64_t tiles = 0;
    for (int32_t i = 0; i < d->n_tensors; ++i) {
        if (d->numel[i] < 0 || d->numel[i] > (std::numeric_limits<int64_t>::max() >> 4))
            return fail(DDP_ERR_INVALID, tensor(i) + " has a bad size");
        if (!known_type(type_of(d->grad_dtype, i)) || !known_type(type_of(d->param_dtype, i)))
            return fail(DDP_ERR_INVALID, tensor(i) + " has an unknown type");
        if (d->weight_decay && !(d->weight_decay[i] >= 0.0 && std::isfinite(d->weight_decay[i])))
            return fail(DDP_ERR_INVALID, tensor(i) + "'s weight decay must be finite and not negative");
        if (d->numel[i] > 0) tiles += d->numel[i] / kAdamTile + 2;   // at most; the cut shifts them
        if (tiles > kMostTiles) return fail(DDP_ERR_INVALID, "the list has too many elements");
    }
    return DDP_OK;
}

// Bytes the tables of a valid desc take at most, wherever its tensors lie.
size_t table_bytes(const ddp_adamw_desc &d)
{
    size_t segs = 0, tiles = 0;
    for (int32_t i = 0; i < d.n_tensors; ++i)
        if (d.numel[i] > 0) {
            ++segs;
            tiles += size_t(d.numel[i] / kAdamTile) + 2;
        }
    return align_up(segs * sizeof(AdamSeg)) + align_up(tiles * sizeof(int32_t)) + kAlign;
}

struct Range {
    uintptr_t lo, hi;
    int32_t of;         // tensor index, or -1: the workspace
    const char *what;
};

constexpr const char *kGrad = "gradient";   // the one range that is only read

// Gradients may share memory; what is written meets nothing else.
int check_overlap(std::vector<Range> &v)
{
    std::sort(v.begin(), v.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    const auto name = [](const Range &r) { return r.of < 0 ? std::string(r.what) : tensor(r.of) + "'s " + r.what; };
    const Range *read = nullptr, *written = nullptr;   // that reach furthest so far
    for (const Range &r : v) {
        const bool reads = r.what == kGrad;
        for (const Range *q : {written, reads ? nullptr : read})
            if (q && r.lo < q->hi) return fail(DDP_ERR_INVALID, name(*q) + " and " + name(r) + " overlap");
        const Range *&furthest = reads ? read : written;
        if (!furthest || furthest->hi < r.hi) furthest = &r;
    }
    return DDP_OK;
}

// Of the sorted ranges those that a step writes; touching ones become one.
Spans written_of(const std::vector<Range> &v)
{
    Spans s;
    for (const Range &r : v) {
        if (r.of < 0 || r.what == kGrad) continue;
        if (!s.empty() && s.back().hi == r.lo)
            s.back().hi = r.hi;
        else
            s.push_back({r.lo, r.hi});
    }
    s.shrink_to_fit();
    return s;
}

int out_of(const ddp_adamw_desc &d, int32_t i, ddp::AdamOut *out)
{
    const int32_t param = type_of(d.param_dtype, i);
    if (!d.copies || !d.copies[i]) {
        *out = param == DDP_F32 ? ddp::kParamF32 : param == DDP_BF16 ? ddp::kParamBF16 : ddp::kParamF16;
        return DDP_OK;
    }
    if (param != DDP_F32 || (d.copy_dtype[i] != DDP_BF16 && d.copy_dtype[i] != DDP_F16))
        return fail(DDP_ERR_INVALID, tensor(i) + "'s copy must be DDP_BF16 or DDP_F16 beside fp32 parameters");
    *out = d.copy_dtype[i] == DDP_BF16 ? ddp::kParamF32CopyBF16 : ddp::kParamF32CopyF16;
    return DDP_OK;
}

int create(const ddp_adamw_desc *d, ddp_adamw **out)
{
    if (!out) return fail(DDP_ERR_INVALID, "out is NULL");
    int rc = check_sizes(d);
    if (rc != DDP_OK) return rc;
    const bool small = d->state == DDP_STATE_8BIT;
    if (d->n_tensors > 0 && (!d->grads || !d->params || !d->m || !d->v))
        return fail(DDP_ERR_INVALID, "grads, params, m or v is NULL");
    if (d->n_tensors > 0 && ((d->m_scale != nullptr) != small || (d->v_scale != nullptr) != small))
        return fail(DDP_ERR_INVALID, "m_scale and v_scale go with 8-bit states");
    const size_t need = table_bytes(*d);
    if (!d->workspace || d->workspace_bytes < need || reinterpret_cast<uintptr_t>(d->workspace) % kAlign)
        return fail(DDP_ERR_INVALID,
                    "workspace missing, misaligned or smaller than " + std::to_string(need) + " bytes");
    const uintptr_t at = reinterpret_cast<uintptr_t>(d->workspace);
    std::vector<Range> ranges{{at, at + need, -1, "the workspace"}};
    std::vector<AdamSeg> segs;
    std::vector<int32_t> tile_seg;
    for (int32_t i = 0; i < d->n_tensors; ++i) {
        const int64_t n = d->numel[i];
        if (n == 0) continue;
        AdamSeg s{};
        s.type = uint8_t(type_of(d->grad_dtype, i));
        rc = out_of(*d, i, &s.out);
        const auto take = [&](const void *p, int size, int64_t count, const char *what) {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
            if (rc != DDP_OK) return;
            if (!lo)
                rc = fail(DDP_ERR_INVALID, tensor(i) + "'s " + what + " is NULL");
            else if (lo % uintptr_t(size))
                rc = fail(DDP_ERR_INVALID, tensor(i) + "'s " + what + " is misaligned for its type");
            else
                ranges.push_back({lo, lo + uintptr_t(size) * uintptr_t(count), i, what});
        };
        const int param_size = element_size(type_of(d->param_dtype, i));
        s.grad = d->grads[i];
        s.param = d->params[i];
        s.m = d->m[i];
        s.v = d->v[i];
        take(s.grad, element_size(s.type), n, kGrad);
        take(s.param, param_size, n, "parameter");
        take(s.m, small ? 1 : 4, n, "m");
        take(s.v, small ? 1 : 4, n, "v");
        if (s.out == ddp::kParamF32CopyBF16 || s.out == ddp::kParamF32CopyF16) {
            s.copy = d->copies[i];
            take(s.copy, 2, n, "copy");
        }
        if (small) {
            const int64_t blocks = (n + kStateBlock - 1) / kStateBlock;
            s.m_scale = d->m_scale[i];
            s.v_scale = d->v_scale[i];
            take(s.m_scale, 4, blocks, "m_scale");
            take(s.v_scale, 4, blocks, "v_scale");
        }
        if (rc != DDP_OK) return rc;
        s.len = n;
        s.decay = d->weight_decay ? d->weight_decay[i] : 0.0;
        s.shift = small ? int16_t(0) : int16_t(reinterpret_cast<uintptr_t>(s.param) % 256 / uintptr_t(param_size));
        s.tile0 = int32_t(tile_seg.size());
        tile_seg.insert(tile_seg.end(), size_t((n + s.shift + kAdamTile - 1) / kAdamTile), int32_t(segs.size()));
        segs.push_back(s);
    }
    rc = check_overlap(ranges);
    if (rc != DDP_OK) return rc;

    std::unique_ptr<ddp_adamw> o(new ddp_adamw());
    o->written = written_of(ranges);
    hipError_t e = hipGetDevice(&o->device);
    if (e != hipSuccess) return hip_fail("device of the AdamW step", e);
    const size_t segs_bytes = align_up(segs.size() * sizeof(AdamSeg));
    std::vector<uint8_t> host(segs_bytes + tile_seg.size() * sizeof(int32_t));
    if (!segs.empty()) {
        std::memcpy(host.data(), segs.data(), segs.size() * sizeof(AdamSeg));
        std::memcpy(host.data() + segs_bytes, tile_seg.data(), tile_seg.size() * sizeof(int32_t));
        e = hipMemcpy(d->workspace, host.data(), host.size(), hipMemcpyHostToDevice);
        if (e != hipSuccess) return hip_fail("workspace upload", e);
    }
    uint8_t *ws = static_cast<uint8_t *>(d->workspace);
    o->tables.segs = reinterpret_cast<const AdamSeg *>(ws);
    o->tables.tile_seg = reinterpret_cast<const int32_t *>(ws + segs_bytes);
    o->tables.tiles = int32_t(tile_seg.size());
    o->tables.bits = small ? 8 : 32;
    *out = o.release();
    return DDP_OK;
}

// What every workgroup reads while others write already.
int check_read(const ddp_adamw *o, const char *what, const void *p, uintptr_t size)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (!p) return DDP_OK;
    if (at % size) return fail(DDP_ERR_INVALID, std::string(what) + " is misaligned");
    if (meets(o->written, at, at + size)) return fail(DDP_ERR_INVALID, std::string(what) + " lies where the step writes");
    return DDP_OK;
}

bool bad_rate(double x)   // of a moment
{
    return !(x >= 0.0 && x < 1.0);
}

bool bad_size(double x)
{
    return !(x >= 0.0 && std::isfinite(x));
}

int step(const ddp_adamw *o, const ddp_adamw_args *a, hipStream_t s)
{
    if (!o || !a) return fail(DDP_ERR_INVALID, "NULL argument");
    if (!a->lr_ptr && bad_size(a->lr)) return fail(DDP_ERR_INVALID, "lr must be finite and not negative");
    // the divisor of an element without a gradient: a subnormal one has no
    // reciprocal in fp32
    if (a->eps != 0.0 && !std::isnormal(float(a->eps)))
        return fail(DDP_ERR_INVALID, "eps must be 0 or a normal fp32 number");
    if (a->eps < 0.0) return fail(DDP_ERR_INVALID, "eps must not be negative");
    // the short quotient takes divisors of up to 2^126; sqrt(v) * root stays below 2^91
    if (o->tables.bits == 8 && a->eps > 0x1p125) return fail(DDP_ERR_INVALID, "eps with 8-bit states must be at most 2^125");
    if (bad_rate(a->beta1) || bad_rate(a->beta2)) return fail(DDP_ERR_INVALID, "beta1 and beta2 must be in [0, 1)");
    if (!a->step_ptr && a->step < 1) return fail(DDP_ERR_INVALID, "step counts from 1");
    if (a->norm && !(a->max_norm >= 0.0f)) return fail(DDP_ERR_INVALID, "max_norm must not be negative");
    if (a->skip_nonfinite && !a->norm) return fail(DDP_ERR_INVALID, "skip_nonfinite needs a norm");
    int rc = check_read(o, "norm", a->norm, sizeof(float));
    if (rc == DDP_OK) rc = check_read(o, "lr_ptr", a->lr_ptr, sizeof(float));
    if (rc == DDP_OK) rc = check_read(o, "step_ptr", a->step_ptr, sizeof(int64_t));
    if (rc != DDP_OK) return rc;
    int now = -1;
    hipError_t e = hipGetDevice(&now);
    if (e != hipSuccess) return hip_fail("current device", e);
    if (now != o->device)
        return fail(DDP_ERR_INVALID, "the AdamW step is on device " + std::to_string(o->device) +
                                         ", the current device is " + std::to_string(now));
    rc = ddp::check_stream(s, now);
    if (rc != DDP_OK || o->tables.tiles == 0) return rc;

    AdamArgs k{};
    k.lr = a->lr;
    k.beta1 = a->beta1;
    k.beta2 = a->beta2;
    k.b1 = float(a->beta1);
    k.a1 = float(1.0 - a->beta1);
    k.b2 = float(a->beta2);
    k.a2 = float(1.0 - a->beta2);
    k.eps = float(a->eps);
    if (!a->lr_ptr && !a->step_ptr) {
        k.size = float(a->lr / (1.0 - ddp::power(a->beta1, a->step)));
        k.root = float(1.0 / std::sqrt(1.0 - ddp::power(a->beta2, a->step)));
    }
    k.max_norm = a->max_norm;
    k.step = a->step;
    k.norm = a->norm;
    k.lr_ptr = a->lr_ptr;
    k.step_ptr = a->step_ptr;
    k.skip = a->skip_nonfinite != 0;
    e = ddp::launch_adamw(o->tables, k, s);
    return e == hipSuccess ? int(DDP_OK) : hip_fail("AdamW step", e);
}

}  // namespace

extern "C" {

size_t ddp_adamw_workspace_bytes(const ddp_adamw_desc *desc)
{
    size_t n = 0;
    guarded([&] {
        const int rc = check_sizes(desc);
        if (rc == DDP_OK) n = table_bytes(*desc);
        return rc;
    });
    return n;
}

int ddp_adamw_create(const ddp_adamw_desc *desc, ddp_adamw **out)
{
    return guarded([&] { return create(desc, out); });
}

int ddp_adamw_destroy(ddp_adamw *o)
{
    delete o;
    return DDP_OK;
}

int ddp_adamw_step(const ddp_adamw *o, const ddp_adamw_args *args, void *stream)
{
    return guarded([&] { return step(o, args, ddp::stream_of(stream)); });
}

}  // extern "C"
