// The norm of a gradient list and its clipping.
//
//   norm = sqrt(sum g^2) | sum |g| | max |g|     over every element of the list
//   f    = min(1, max_norm / (norm + 1e-6))      (NaN stays NaN)
//   out  = R(g * f)                              R: one rounding to the output's type
//
// Two passes over HBM and few operations an element (one conversion and one
// fused multiply-add), so both passes are bound by memory; the second cannot
// begin before the first has ended. 953M bf16 elements: the norm 275 us (6.9
// TB/s), scaling them into fp32 949 us (6.0 TB/s).
//
//   * Sums are held in 64 bits from the first element on: a product of two
//     fp32 values is exact there and cannot overflow or vanish, and a billion
//     terms lose nothing an fp32 result could show. The vector ALU's fp64
//     rate leaves room: two fp64 operations an element.
//   * max |g| is taken on the bit patterns of |g| as unsigned integers, where
//     a NaN is above every number: it stays in the result as in a sum.
//   * Every order is fixed: a thread's elements, the threads of a wave, the
//     waves of a workgroup, the workgroups' partials. No atomics; a list gives
//     the same bits every time.
//   * Lists of many tiles that go into other buffers finish the norm in a
//     launch of its own. Otherwise the workgroups of the clipping pass, at most
//     eight a CU, each reduce the partials for themselves (at most 8 KiB from
//     L2) instead of waiting for such a launch.
#include "../../include/ddp.h"
#include "element.h"
#include "grad_list.h"

#include <hip/hip_runtime.h>

namespace ddp {
namespace {

// Vectors are read and written past the caches, in the norm too, though the
// clipping pass reads the same data again: 953M bf16 elements 287 us against
// 313 (335M fp32 195 against 221), and the clipping after it took the same
// time either way, or less.
template <int TYPE, int VEC>
__device__ __forceinline__ typename Raw<TYPE, VEC>::type load(const void *p, int64_t e)
{
    return __builtin_nontemporal_load(
        (const GLOBAL typename Raw<TYPE, VEC>::any *)(static_cast<const typename Raw<TYPE, VEC>::elem *>(p) + e));
}

template <int TYPE, int VEC>
__device__ __forceinline__ void store(void *p, int64_t e, const typename Raw<TYPE, VEC>::type &v)
{
    __builtin_nontemporal_store(
        v, (GLOBAL typename Raw<TYPE, VEC>::any *)(static_cast<typename Raw<TYPE, VEC>::elem *>(p) + e));
}

template <int TYPE>
__device__ __forceinline__ float load1(const void *p, int64_t e)
{
    return widen<TYPE>(((const GLOBAL typename Raw<TYPE, 1>::elem *)p)[e]);
}

// Elements of a tile that its tensor has: whole vectors lie in [body, end) of
// it, the few before and after go one a thread.
struct Part {
    int lo, body, end, hi;   // offsets in the tile
};

__device__ __forceinline__ Part part_of(int64_t base, int64_t len, int span, int vec)
{
    Part p;
    p.hi = int(max(int64_t(0), min(int64_t(span), len - base)));
    p.lo = base < 0 ? min(p.hi, int(-base)) : 0;
    p.body = min(p.hi, (p.lo + vec - 1) / vec * vec);
    p.end = max(p.body, p.hi / vec * vec);
    return p;
}

// The element of the part before the body, or after it, that thread t has, or
// -1.
__device__ __forceinline__ int odd_element(const Part &p, int t)
{
    if (t < p.body - p.lo) return p.lo + t;
    t -= 64;
    return t >= 0 && t < p.hi - p.end ? p.end + t : -1;
}

// The running value of a norm. A thread keeps four of them for the four
// elements of a vector, so that successive additions do not wait for each
// other.
template <int NORM>
struct Running {
    double a[4] = {0.0, 0.0, 0.0, 0.0};
    __device__ __forceinline__ void add(int j, float x)
    {
        if (NORM == DDP_NORM_L2)
            a[j] = __fma_rn(double(x), double(x), a[j]);
        else
            a[j] += double(fabsf(x));
    }
    __device__ __forceinline__ double value() const { return (a[0] + a[1]) + (a[2] + a[3]); }
    static __device__ __forceinline__ double merge(double x, double y) { return x + y; }
};

template <>
struct Running<DDP_NORM_INF> {
    uint32_t a = 0;
    __device__ __forceinline__ void add(int, float x) { a = max(a, __float_as_uint(x) & 0x7fffffffu); }
    __device__ __forceinline__ double value() const { return __hiloint2double(0, int(a)); }
    static __device__ __forceinline__ double merge(double x, double y)
    {
        return uint32_t(__double2loint(x)) >= uint32_t(__double2loint(y)) ? x : y;
    }
};

// The norm from the merged partials, rounded to fp32 once.
template <int NORM>
__device__ __forceinline__ float finished(double v)
{
    if (NORM == DDP_NORM_INF) return __uint_as_float(uint32_t(__double2loint(v)));
    return float(NORM == DDP_NORM_L2 ? __dsqrt_rn(v) : v);
}

// Every thread gets the workgroup's merged value.
template <int NORM, int THREADS>
__device__ __forceinline__ double over_workgroup(double v)
{
    __shared__ double wave[THREADS / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = Running<NORM>::merge(v, __shfl_xor(v, d));
    __syncthreads();   // an earlier use of `wave` has been read
    if (threadIdx.x % 64 == 0) wave[threadIdx.x / 64] = v;
    __syncthreads();
    v = wave[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v = Running<NORM>::merge(v, wave[w]);
    return v;
}

template <int NORM, int THREADS>
__device__ __forceinline__ double merged_partials(const double *partials, int n)
{
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += THREADS) v = Running<NORM>::merge(v, ((const GLOBAL double *)partials)[i]);
    return over_workgroup<NORM, THREADS>(v);
}

// One tile into the running norm. All loads of a thread are issued before the
// first value is used.
template <int NORM, int TYPE, int THREADS>
__device__ __forceinline__ void norm_tile(const GradSeg &s, int64_t base, int tid, Running<NORM> &r)
{
    constexpr int VEC = TYPE == DDP_F32 ? 4 : 8;   // 16 bytes
    constexpr int SPAN = kGradTile, U = SPAN / (THREADS * VEC);
    typename Raw<TYPE, VEC>::type x[U];
    const int o = tid * VEC;
    if (base >= 0 && base + kGradTile <= s.len) {
#pragma unroll
        for (int k = 0; k < U; ++k) x[k] = load<TYPE, VEC>(s.src, base + o + k * THREADS * VEC);
    } else {
        const Part p = part_of(base, s.len, SPAN, VEC);
        const int odd = odd_element(p, tid);
        const float y = odd >= 0 ? load1<TYPE>(s.src, base + odd) : 0.0f;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int at = o + k * THREADS * VEC;
            x[k] = 0;
            if (at >= p.body && at < p.end) x[k] = load<TYPE, VEC>(s.src, base + at);
        }
        r.add(0, y);
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) r.add(j % 4, widen<TYPE>(x[k][j]));
}

template <int IN, int OUT, int THREADS, int SPAN>
__device__ __forceinline__ void clip_tile(const GradSeg &s, int64_t base, int tid, float f)
{
    constexpr int VEC = IN == DDP_F32 || OUT == DDP_F32 ? 4 : 8;   // 16 bytes of the wider type
    constexpr int U = SPAN / (THREADS * VEC);
    typename Raw<IN, VEC>::type x[U];
    const int o = tid * VEC;
    const auto scaled = [f](const typename Raw<IN, VEC>::type &v) {
        typename Raw<OUT, VEC>::type y;
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[j] = narrow<OUT>(__fmul_rn(widen<IN>(v[j]), f));
        return y;
    };
    if (base >= 0 && base + SPAN <= s.len) {
#pragma unroll
        for (int k = 0; k < U; ++k) x[k] = load<IN, VEC>(s.src, base + o + k * THREADS * VEC);
#pragma unroll
        for (int k = 0; k < U; ++k) store<OUT, VEC>(s.dst, base + o + k * THREADS * VEC, scaled(x[k]));
        return;
    }
    const Part p = part_of(base, s.len, SPAN, VEC);
    const int odd = odd_element(p, tid);
    const float y = odd >= 0 ? load1<IN>(s.src, base + odd) : 0.0f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int at = o + k * THREADS * VEC;
        if (at >= p.body && at < p.end) x[k] = load<IN, VEC>(s.src, base + at);
    }
    if (odd >= 0) ((GLOBAL typename Raw<OUT, 1>::elem *)s.dst)[base + odd] = narrow<OUT>(__fmul_rn(y, f));
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int at = o + k * THREADS * VEC;
        if (at >= p.body && at < p.end) store<OUT, VEC>(s.dst, base + at, scaled(x[k]));
    }
}

__device__ __forceinline__ GradSeg seg_of(const GradTables &t, int tile)
{
    typedef uint32_t words __attribute__((ext_vector_type(8)));
    typedef words any __attribute__((aligned(16)));   // as the workspace is
    const int k = ((const CONSTANT int32_t *)t.tile_seg)[tile];
    const words w = ((const CONSTANT any *)t.segs)[k];
    return __builtin_bit_cast(GradSeg, w);
}

template <int NORM, int THREADS>
__device__ __forceinline__ void norm_any(const GradSeg &s, int tile, int tid, Running<NORM> &r)
{
    const int64_t base = int64_t(tile - s.tile0) * kGradTile - s.shift;
    if (s.in == DDP_F32)
        norm_tile<NORM, DDP_F32, THREADS>(s, base, tid, r);
    else if (s.in == DDP_BF16)
        norm_tile<NORM, DDP_BF16, THREADS>(s, base, tid, r);
    else
        norm_tile<NORM, DDP_F16, THREADS>(s, base, tid, r);
}

template <int IN, int THREADS, int SPAN>
__device__ __forceinline__ void clip_out(const GradSeg &s, int64_t base, int tid, float f)
{
    if (s.out == DDP_F32)
        clip_tile<IN, DDP_F32, THREADS, SPAN>(s, base, tid, f);
    else if (s.out == DDP_BF16)
        clip_tile<IN, DDP_BF16, THREADS, SPAN>(s, base, tid, f);
    else
        clip_tile<IN, DDP_F16, THREADS, SPAN>(s, base, tid, f);
}

// Part `sub` of a tile, SPAN elements of it.
template <int THREADS, int SPAN>
__device__ __forceinline__ void clip_any(const GradSeg &s, int tile, int sub, int tid, float f)
{
    const int64_t base = int64_t(tile - s.tile0) * kGradTile - s.shift + sub * SPAN;
    if (s.in == DDP_F32)
        clip_out<DDP_F32, THREADS, SPAN>(s, base, tid, f);
    else if (s.in == DDP_BF16)
        clip_out<DDP_BF16, THREADS, SPAN>(s, base, tid, f);
    else
        clip_out<DDP_F16, THREADS, SPAN>(s, base, tid, f);
}

constexpr int kNormThreads = 256;
constexpr int kSmallThreads = 1024;

template <int NORM>
__global__ void __launch_bounds__(kNormThreads) norm_partials(GradTables t, double *partials)
{
    Running<NORM> r;
    int tile = blockIdx.x;
    GradSeg s{};
    if (tile < t.norm_tiles) s = seg_of(t, tile);
    while (tile < t.norm_tiles) {
        const int next = tile + int(gridDim.x);
        const GradSeg after = next < t.norm_tiles ? seg_of(t, next) : s;   // arrives behind this tile's loads
        norm_any<NORM, kNormThreads>(s, tile, int(threadIdx.x), r);
        tile = next;
        s = after;
    }
    const double v = over_workgroup<NORM, kNormThreads>(r.value());
    if (threadIdx.x == 0) ((GLOBAL double *)partials)[blockIdx.x] = v;
}

template <int NORM>
__global__ void __launch_bounds__(kSmallThreads) norm_finish(int n, const double *partials, float *norm)
{
    const double v = merged_partials<NORM, kSmallThreads>(partials, n);
    if (threadIdx.x == 0) *(GLOBAL float *)norm = finished<NORM>(v);
}

template <int NORM>
__global__ void __launch_bounds__(kNormThreads)
clip_all(GradTables t, ClipFactor c, int n_partials, const double *partials, float *norm)
{
    float n;
    if (c.norm) {
        n = *(const CONSTANT float *)c.norm;
    } else {
        n = finished<NORM>(merged_partials<NORM, kNormThreads>(partials, n_partials));
        if (blockIdx.x == 0 && threadIdx.x == 0) *(GLOBAL float *)norm = n;
    }
    const float f = clip_factor(c.max_norm, n);
    if (f == 1.0f && t.in_place) return;   // x * 1 is x
    // from the last tile down: the norm's pass left those in the caches
    for (int tile = t.all_tiles - 1 - int(blockIdx.x); tile >= 0; tile -= int(gridDim.x))
        clip_any<kNormThreads, kGradTile>(seg_of(t, tile), tile, 0, int(threadIdx.x), f);
}

// A part of a tile a workgroup, with the norm given: 953M elements from bf16
// into fp32 956 us (6.0 TB/s), against 986 with parts of 4096, 1001 with whole
// tiles and 1057 with workgroups that go from tile to tile.
constexpr int kClipSpan = 2048;

__global__ void __launch_bounds__(kNormThreads) clip_parts(GradTables t, ClipFactor c)
{
    constexpr int PARTS = kGradTile / kClipSpan;
    const int part = t.all_tiles * PARTS - 1 - int(blockIdx.x);
    const int tile = part / PARTS;
    const GradSeg s = seg_of(t, tile);
    clip_any<kNormThreads, kClipSpan>(s, tile, part % PARTS, int(threadIdx.x),
                                      clip_factor(c.max_norm, *(const CONSTANT float *)c.norm));
}

// Four groups of 256 threads, each with every fourth tile.
template <int NORM, bool CLIP>
__global__ void __launch_bounds__(kSmallThreads) small_list(GradTables t, float max_norm, float *norm)
{
    constexpr int GROUPS = kSmallThreads / kNormThreads;
    const int group = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kNormThreads);
    const int tid = int(threadIdx.x) % kNormThreads;
    Running<NORM> r;
    for (int tile = group; tile < t.norm_tiles; tile += GROUPS)
        norm_any<NORM, kNormThreads>(seg_of(t, tile), tile, tid, r);
    const float n = finished<NORM>(over_workgroup<NORM, kSmallThreads>(r.value()));
    if (threadIdx.x == 0) *(GLOBAL float *)norm = n;
    if (!CLIP) return;
    const float f = clip_factor(max_norm, n);
    if (f == 1.0f && t.in_place) return;
    for (int tile = group; tile < t.all_tiles; tile += GROUPS)
        clip_any<kNormThreads, kGradTile>(seg_of(t, tile), tile, 0, tid, f);
}

}  // namespace

hipError_t launch_norm_partials(int norm_type, const GradTables &t, int blocks, void *partials, hipStream_t s)
{
    double *p = static_cast<double *>(partials);
    const dim3 g(blocks), b(kNormThreads);
    switch (norm_type) {
    case DDP_NORM_L1: hipLaunchKernelGGL((norm_partials<DDP_NORM_L1>), g, b, 0, s, t, p); break;
    case DDP_NORM_L2: hipLaunchKernelGGL((norm_partials<DDP_NORM_L2>), g, b, 0, s, t, p); break;
    default: hipLaunchKernelGGL((norm_partials<DDP_NORM_INF>), g, b, 0, s, t, p); break;
    }
    return hipGetLastError();
}

hipError_t launch_norm_finish(int norm_type, int blocks, const void *partials, float *norm, hipStream_t s)
{
    const double *p = static_cast<const double *>(partials);
    const dim3 g(1), b(kSmallThreads);
    switch (norm_type) {
    case DDP_NORM_L1: hipLaunchKernelGGL((norm_finish<DDP_NORM_L1>), g, b, 0, s, blocks, p, norm); break;
    case DDP_NORM_L2: hipLaunchKernelGGL((norm_finish<DDP_NORM_L2>), g, b, 0, s, blocks, p, norm); break;
    default: hipLaunchKernelGGL((norm_finish<DDP_NORM_INF>), g, b, 0, s, blocks, p, norm); break;
    }
    return hipGetLastError();
}

hipError_t launch_clip(int norm_type, const GradTables &t, int blocks, const ClipFactor &f, int n_partials,
                       const void *partials, float *norm, hipStream_t s)
{
    const double *p = static_cast<const double *>(partials);
    const dim3 g(blocks), b(kNormThreads);
    switch (norm_type) {
    case DDP_NORM_L1: hipLaunchKernelGGL((clip_all<DDP_NORM_L1>), g, b, 0, s, t, f, n_partials, p, norm); break;
    case DDP_NORM_L2: hipLaunchKernelGGL((clip_all<DDP_NORM_L2>), g, b, 0, s, t, f, n_partials, p, norm); break;
    default: hipLaunchKernelGGL((clip_all<DDP_NORM_INF>), g, b, 0, s, t, f, n_partials, p, norm); break;
    }
    return hipGetLastError();
}

hipError_t launch_clip_parts(const GradTables &t, const ClipFactor &f, hipStream_t s)
{
    const dim3 g(static_cast<unsigned>(t.all_tiles) * (kGradTile / kClipSpan)), b(kNormThreads);
    hipLaunchKernelGGL(clip_parts, g, b, 0, s, t, f);
    return hipGetLastError();
}

template <int NORM>
static void run_small(const GradTables &t, bool clip, float max_norm, float *norm, hipStream_t s)
{
    const dim3 g(1), b(kSmallThreads);
    if (clip)
        hipLaunchKernelGGL((small_list<NORM, true>), g, b, 0, s, t, max_norm, norm);
    else
        hipLaunchKernelGGL((small_list<NORM, false>), g, b, 0, s, t, max_norm, norm);
}

hipError_t launch_small(int norm_type, const GradTables &t, bool clip, float max_norm, float *norm, hipStream_t s)
{
    switch (norm_type) {
    case DDP_NORM_L1: run_small<DDP_NORM_L1>(t, clip, max_norm, norm, s); break;
    case DDP_NORM_L2: run_small<DDP_NORM_L2>(t, clip, max_norm, norm, s); break;
    default: run_small<DDP_NORM_INF>(t, clip, max_norm, norm, s); break;
    }
    return hipGetLastError();
}

}  // namespace ddp
