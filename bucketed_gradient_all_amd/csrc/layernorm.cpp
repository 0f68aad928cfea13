// Host half of the layer norm: validation, the workspace's layout and the
// launches.
#include "layernorm.h"
#include "host_common.h"
#include "spans.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <vector>

using ddp::fail;
using ddp::guarded;
using ddp::hip_fail;
using ddp::LayerArgs;
using ddp::LayerBackward;
using ddp::LayerForward;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMostColumns = int64_t(1) << 26;

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

// Bytes of z from which rows are read past the caches; below, they may still lie
// there from the kernel before. 128 MiB forward 85.5 us against 87.2, backward 97
// against 100; 64 MiB forward 44.7 us against 45.6 from memory, but 44 against 40
// where the caches hold a part.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

int element_size(int32_t type)
{
    return type == DDP_F32 ? 4 : 2;
}

bool known_type(int32_t type)
{
    return type == DDP_F32 || type == DDP_BF16 || type == DDP_F16;
}

int check_desc(const ddp_layernorm_desc *d, int64_t n_rows)
{
    if (!d) return fail(DDP_ERR_INVALID, "desc is NULL");
    if (d->width < 0 || d->width > kMostColumns) return fail(DDP_ERR_INVALID, "width must be in [0, 2^26]");
    if (d->kind != DDP_LAYER_NORM && d->kind != DDP_RMS_NORM)
        return fail(DDP_ERR_INVALID, "unknown kind " + std::to_string(d->kind));
    if (!known_type(d->x_dtype) || !known_type(d->y_dtype) || !known_type(d->weight_dtype) || !known_type(d->grad_dtype))
        return fail(DDP_ERR_INVALID, "unknown element type in the desc");
    if (d->x_dtype != DDP_F32 && d->y_dtype != d->x_dtype)
        return fail(DDP_ERR_INVALID, "y_dtype must be x_dtype unless that is DDP_F32");
    if (!(d->eps >= 0.0f) || std::isinf(d->eps)) return fail(DDP_ERR_INVALID, "eps must be finite and not negative");
    for (int64_t s : {d->x_stride, d->add_stride, d->z_stride, d->y_stride})
        if (s < 0 || s > (int64_t(1) << 31)) return fail(DDP_ERR_INVALID, "strides must be in [0, 2^31]");
    if (n_rows < 0 || n_rows >= (int64_t(1) << 31)) return fail(DDP_ERR_INVALID, "n_rows must be in [0, 2^31)");
    if (std::max({d->x_stride, d->add_stride, d->z_stride, d->y_stride}) * n_rows > int64_t(1) << 58)
        return fail(DDP_ERR_INVALID, "n_rows times a stride is too large");
    return DDP_OK;
}

// Whether rows are read past the caches.
bool streams(const ddp_layernorm_desc &d, int64_t n_rows)
{
    return n_rows > kStreamBytes / (std::max<int64_t>(1, d.width) * element_size(d.x_dtype));
}

LayerArgs args_of(const ddp_layernorm_desc &d, int64_t n_rows)
{
    LayerArgs a{};
    a.rows = n_rows;
    a.width = d.width;
    a.x_stride = d.x_stride;
    a.add_stride = d.add_stride;
    a.z_stride = d.z_stride;
    a.y_stride = d.y_stride;
    a.eps = d.eps;
    a.rms = d.kind == DDP_RMS_NORM;
    a.stream = streams(d, n_rows);
    a.x_dtype = d.x_dtype;
    a.y_dtype = d.y_dtype;
    a.weight_dtype = d.weight_dtype;
    a.grad_dtype = d.grad_dtype;
    return a;
}

// An argument: n rows of `bytes` bytes, `stride` bytes apart.
struct Operand {
    const char *name;
    const void *p;
    int64_t n, stride, bytes;
    int align;
    uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t hi() const { return lo() + uintptr_t((n - 1) * stride + bytes); }
    bool one_range() const { return n == 1 || stride <= bytes; }
};

Operand rows(const char *name, const void *p, int64_t n, int64_t stride, int64_t width, int32_t type)
{
    const int size = element_size(type);
    return {name, p, stride == 0 ? 1 : n, stride * size, width * size, size};
}

Operand line(const char *name, const void *p, int64_t n, int size)
{
    return {name, p, 1, n * size, n * size, size};
}

// Rows of one stride that interleave are apart; of two strides they are taken
// to meet where their ranges do.
bool meet(const Operand &a, const Operand &b)
{
    if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    if (a.one_range()) return ddp::rows_meet(b.p, b.n, b.stride, b.bytes, a.lo(), a.hi());
    if (b.one_range()) return ddp::rows_meet(a.p, a.n, a.stride, a.bytes, b.lo(), b.hi());
    if (a.stride != b.stride) return true;
    const bool first = a.lo() <= b.lo();
    const int64_t off = int64_t((first ? b.lo() - a.lo() : a.lo() - b.lo()) % uintptr_t(a.stride));
    return off < (first ? a : b).bytes || a.stride - off < (first ? b : a).bytes;
}

bool same_place(const Operand &a, const Operand &b)
{
    return a.p == b.p && a.n == b.n && (a.n == 1 || a.stride == b.stride) && a.bytes == b.bytes && a.align == b.align;
}

int check_pointer(const Operand &o)
{
    if (!o.p) return fail(DDP_ERR_INVALID, std::string(o.name) + " is NULL");
    if (o.lo() % uintptr_t(o.align)) return fail(DDP_ERR_INVALID, std::string(o.name) + " is misaligned");
    return DDP_OK;
}

// Pointers that are there and aligned, and outputs that meet no other argument,
// but for those of `instead` that may lie exactly where one of `of` does.
int check_operands(const std::vector<Operand> &in, const std::vector<Operand> &out,
                   std::initializer_list<const char *> instead, std::initializer_list<const char *> of)
{
    const auto among = [](std::initializer_list<const char *> names, const char *name) {
        return std::find(names.begin(), names.end(), name) != names.end();
    };
    for (const auto *v : {&in, &out})
        for (const Operand &o : *v)
            if (const int rc = check_pointer(o)) return rc;
    for (size_t i = 0; i < out.size(); ++i) {
        for (const Operand &o : in) {
            if (among(instead, out[i].name) && among(of, o.name) && same_place(out[i], o)) continue;
            if (meet(out[i], o)) return fail(DDP_ERR_INVALID, std::string(out[i].name) + " and " + o.name + " overlap");
        }
        for (size_t k = 0; k < i; ++k)
            if (meet(out[i], out[k]))
                return fail(DDP_ERR_INVALID, std::string(out[k].name) + " and " + out[i].name + " overlap");
    }
    return DDP_OK;
}

// The names that check_operands compares, each one object.
constexpr char kX[] = "x", kAdd[] = "add", kZ[] = "z", kY[] = "y", kDy[] = "dy", kDz[] = "dz", kDx[] = "dx";

int check_device(hipStream_t s)
{
    int now = -1;
    const hipError_t e = hipGetDevice(&now);
    if (e != hipSuccess) return hip_fail("current device", e);
    return ddp::check_stream(s, now);
}

int forward(const ddp_layernorm_desc *d, int64_t n, const LayerForward &f, hipStream_t s)
{
    int rc = check_desc(d, n);
    if (rc != DDP_OK) return rc;
    if (f.z && !f.add) return fail(DDP_ERR_INVALID, "z is given without add");
    if (n > 1 && (d->x_stride < d->width || d->y_stride < d->width || (f.z && d->z_stride < d->width)))
        return fail(DDP_ERR_INVALID, "strides of x, z and y must be at least the width");
    if (n == 0 || d->width == 0) return DDP_OK;
    std::vector<Operand> in{rows(kX, f.x, n, d->x_stride, d->width, d->x_dtype)};
    if (f.add) in.push_back(rows(kAdd, f.add, n, d->add_stride, d->width, d->x_dtype));
    if (f.weight) in.push_back(line("weight", f.weight, d->width, element_size(d->weight_dtype)));
    if (f.bias) in.push_back(line("bias", f.bias, d->width, element_size(d->weight_dtype)));
    std::vector<Operand> out{rows(kY, f.y, n, d->y_stride, d->width, d->y_dtype)};
    if (f.z) out.push_back(rows(kZ, f.z, n, d->z_stride, d->width, d->x_dtype));
    if (f.mean) out.push_back(line("mean", f.mean, n, 4));
    if (f.rstd) out.push_back(line("rstd", f.rstd, n, 4));
    rc = check_operands(in, out, {kY, kZ}, {kX, kAdd});
    if (rc == DDP_OK) rc = check_device(s);
    if (rc != DDP_OK) return rc;
    const hipError_t e = ddp::launch_layernorm(args_of(*d, n), f, s);
    return e == hipSuccess ? int(DDP_OK) : hip_fail("layer norm", e);
}

// How the gradient's workgroups share the rows.
struct Plan {
    bool wide;         // rows are read again instead of held in registers
    int32_t n_parts;   // workgroups along the rows
    size_t bytes;      // of the workspace
};

// Parts at most: eight waves on each of 256 CUs, or nine where they are three a
// workgroup, so that every CU has as many.
constexpr int64_t kMostThreads = int64_t(512) * 256;

Plan plan_of(const ddp_layernorm_desc &d, int64_t n_rows)
{
    Plan p{};
    const int64_t vec = ddp::layer_vector(d.x_dtype, d.y_dtype);
    const int64_t vectors = std::max<int64_t>(1, ceil_div(d.width, vec));
    p.wide = vectors > ddp::kRowVectors;
    const ddp::RowPlan r = ddp::row_plan(vectors, vec, streams(d, n_rows));
    int64_t most = ceil_div(kMostThreads / r.threads, 256) * 256, rows = r.rows;
    if (p.wide) most = std::max<int64_t>(1, 1024 / ceil_div(vectors, 64)), rows = 4;
    p.n_parts = int32_t(std::min(most, ceil_div(n_rows, rows)));
    p.bytes = (size_t(p.n_parts) * 2 * size_t(d.width) * sizeof(float) + kAlign - 1) / kAlign * kAlign + kAlign;
    return p;
}

// Rows, bytes of z and dy, and their product of a call that goes in one launch, at
// most. Replayed from a graph, one launch against two: 64 rows of 1024 16-bit
// columns 4.0 us against 7.1, 1024 rows 5.1 against 8.6, 1024 rows of 2047 8.3
// against 11.7, 256 rows of 8192 6.0 against 16.7; the other side, where a
// workgroup goes over all rows of its columns: 2048 rows of 64 7.5 against 6.5, of
// 1024 fp32 columns 15.4 against 9.7. Called one by one, the host saves 3 us too.
constexpr int64_t kSmallRows = 2048, kSmallBytes = int64_t(8) << 20, kSmallWork = int64_t(1) << 33;

bool is_small(const ddp_layernorm_desc &d, int64_t n, const LayerBackward &b, const Plan &p)
{
    if (n == 0 || n > kSmallRows || p.wide || b.dx == b.dy) return false;
    const int64_t bytes = n * d.width * (element_size(d.x_dtype) + element_size(d.y_dtype));
    return bytes <= kSmallBytes && n * bytes <= kSmallWork;
}

int backward(const ddp_layernorm_desc *d, int64_t n, LayerBackward b, void *workspace, size_t workspace_bytes,
             hipStream_t s)
{
    int rc = check_desc(d, n);
    if (rc != DDP_OK) return rc;
    const bool sums = b.dweight || b.dbias;
    if (n > 1 && b.dx && d->x_stride < d->width)
        return fail(DDP_ERR_INVALID, "the stride of dx must be at least the width");
    if (d->width == 0 || (n == 0 && (b.accumulate || !sums)) || (!b.dx && !sums)) return DDP_OK;
    std::vector<Operand> in, out;
    if (n > 0) {
        in.push_back(rows(kDy, b.dy, n, d->y_stride, d->width, d->y_dtype));
        in.push_back(rows(kZ, b.z, n, d->z_stride, d->width, d->x_dtype));
        if (b.dz) in.push_back(rows(kDz, b.dz, n, d->z_stride, d->width, d->x_dtype));
        if (b.weight) in.push_back(line("weight", b.weight, d->width, element_size(d->weight_dtype)));
        if (d->kind == DDP_LAYER_NORM) in.push_back(line("mean", b.mean, n, 4));
        in.push_back(line("rstd", b.rstd, n, 4));
        if (b.dx) out.push_back(rows(kDx, b.dx, n, d->x_stride, d->width, d->x_dtype));
    }
    if (b.dweight) out.push_back(line("dweight", b.dweight, d->width, element_size(d->grad_dtype)));
    if (b.dbias) out.push_back(line("dbias", b.dbias, d->width, element_size(d->grad_dtype)));
    const Plan p = plan_of(*d, n);
    if (sums) {
        if (!workspace || workspace_bytes < p.bytes || reinterpret_cast<uintptr_t>(workspace) % kAlign)
            return fail(DDP_ERR_INVALID,
                        "workspace missing, misaligned or smaller than " + std::to_string(p.bytes) + " bytes");
        out.push_back(line("workspace", workspace, int64_t(p.bytes), 1));
    }
    rc = check_operands(in, out, {kDx}, {kDy, kDz});
    if (rc == DDP_OK) rc = check_device(s);
    if (rc != DDP_OK) return rc;
    const LayerArgs a = args_of(*d, n);
    if (d->kind == DDP_RMS_NORM) b.mean = nullptr;
    b.parts = sums ? static_cast<float *>(workspace) : nullptr;
    b.n_parts = p.n_parts;
    hipError_t e = hipSuccess;
    if (sums && is_small(*d, n, b, p)) {
        e = ddp::launch_layernorm_small(a, b, s);
        return e == hipSuccess ? int(DDP_OK) : hip_fail("layer norm's gradient", e);
    }
    if (n > 0) e = p.wide ? ddp::launch_layernorm_wide(a, b, s) : ddp::launch_layernorm_rows(a, b, s);
    if (e == hipSuccess && sums) e = ddp::launch_layernorm_join(a, b, s);
    return e == hipSuccess ? int(DDP_OK) : hip_fail("layer norm's gradient", e);
}

}  // namespace

extern "C" {

int ddp_layernorm(const ddp_layernorm_desc *desc, int64_t n_rows, const void *x, const void *add, const void *weight,
                  const void *bias, void *z, void *y, float *mean, float *rstd, void *stream)
{
    return guarded([&] {
        return forward(desc, n_rows, LayerForward{x, add, weight, bias, z, y, mean, rstd}, ddp::stream_of(stream));
    });
}

size_t ddp_layernorm_grad_workspace_bytes(const ddp_layernorm_desc *desc, int64_t n_rows)
{
    size_t n = 0;
    guarded([&] {
        const int rc = check_desc(desc, n_rows);
        if (rc == DDP_OK) n = plan_of(*desc, n_rows).bytes;
        return rc;
    });
    return n;
}

int ddp_layernorm_grad(const ddp_layernorm_desc *desc, int64_t n_rows, const void *dy, const void *z, const void *dz,
                       const void *weight, const float *mean, const float *rstd, void *dx, void *dweight, void *dbias,
                       int32_t accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        LayerBackward b{};
        b.dy = dy;
        b.z = z;
        b.dz = dz;
        b.weight = weight;
        b.mean = mean;
        b.rstd = rstd;
        b.dx = dx;
        b.dweight = dweight;
        b.dbias = dbias;
        b.accumulate = accumulate != 0;
        return backward(desc, n_rows, b, workspace, workspace_bytes, ddp::stream_of(stream));
    });
}

}  // extern "C"
