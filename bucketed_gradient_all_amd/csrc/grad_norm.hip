// The norm of a gradient list and its clipping.
//
//   norm = sqrt(sum g^2) | sum |g| | max |g|     over every element of the list
//   f    = min(1, max_norm / (norm + 1e-6))      (NaN stays NaN)
//   out  = R(g * f)                              R: one rounding to the output's type
//
// Two passes over HBM and few operations an element (one conversion and one
// fused multiply-add), so both passes are bound by memory; the second cannot
// begin before the first has ended.
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
//   * The workgroups of the clipping pass each reduce the partials for
//     themselves (at most 16 KiB from L2) instead of waiting for a launch that
//     does it once.
#include "../../include/ddp.h"
#include "grad_list.h"

#include <hip/hip_runtime.h>

namespace ddp {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
// the same at any element's alignment: a list's tensors start where they do,
// and global memory takes vectors at any address
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u16x4 u16x4_any __attribute__((aligned(2)));

#define GLOBAL __attribute__((address_space(1)))

template <int TYPE>
__device__ __forceinline__ float widen(unsigned short h)
{
    if (TYPE == DDP_BF16) return __uint_as_float(uint32_t(h) << 16);
    return float(__builtin_bit_cast(_Float16, h));
}

// One rounding to the type, to nearest even; beyond fp16's range it is inf.
template <int TYPE>
__device__ __forceinline__ unsigned short narrow(float v)
{
    if (TYPE == DDP_BF16) return __builtin_bit_cast(unsigned short, static_cast<__bf16>(v));
    // keeps the product a separately rounded fp32 value (see `wire` in
    // reduce_kernels.h)
    asm volatile("" : "+v"(v));
    return __builtin_bit_cast(unsigned short, static_cast<_Float16>(v));
}

template <int TYPE>
__device__ __forceinline__ f32x4 load4(const void *p, int64_t e)
{
    if (TYPE == DDP_F32) return *(const GLOBAL f32x4_any *)(static_cast<const float *>(p) + e);
    const u16x4 h = *(const GLOBAL u16x4_any *)(static_cast<const unsigned short *>(p) + e);
    return f32x4{widen<TYPE>(h.x), widen<TYPE>(h.y), widen<TYPE>(h.z), widen<TYPE>(h.w)};
}

template <int TYPE>
__device__ __forceinline__ float load1(const void *p, int64_t e)
{
    if (TYPE == DDP_F32) return *(const GLOBAL float *)(static_cast<const float *>(p) + e);
    return widen<TYPE>(*(const GLOBAL unsigned short *)(static_cast<const unsigned short *>(p) + e));
}

template <int TYPE>
__device__ __forceinline__ void store4(void *p, int64_t e, f32x4 v)
{
    if (TYPE == DDP_F32) {
        *(GLOBAL f32x4_any *)(static_cast<float *>(p) + e) = v;
    } else {
        const u16x4 h = {narrow<TYPE>(v.x), narrow<TYPE>(v.y), narrow<TYPE>(v.z), narrow<TYPE>(v.w)};
        *(GLOBAL u16x4_any *)(static_cast<unsigned short *>(p) + e) = h;
    }
}

template <int TYPE>
__device__ __forceinline__ void store1(void *p, int64_t e, float v)
{
    if (TYPE == DDP_F32)
        *(GLOBAL float *)(static_cast<float *>(p) + e) = v;
    else
        *(GLOBAL unsigned short *)(static_cast<unsigned short *>(p) + e) = narrow<TYPE>(v);
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

__device__ __forceinline__ float clip_factor(float max_norm, float norm)
{
    const float f = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
    return f >= 1.0f ? 1.0f : f;
}

// One tile into the running norm.
template <int NORM, int TYPE, int THREADS>
__device__ __forceinline__ void norm_tile(const GradSeg &s, int64_t base, Running<NORM> &r)
{
    constexpr int U = kGradTile / (THREADS * 4);
    const int64_t e0 = base + int(threadIdx.x) * 4;
    if (base >= 0 && base + kGradTile <= s.len) {
        f32x4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) x[k] = load4<TYPE>(s.src, e0 + k * THREADS * 4);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            r.add(0, x[k].x);
            r.add(1, x[k].y);
            r.add(2, x[k].z);
            r.add(3, x[k].w);
        }
        return;
    }
    for (int k = 0; k < U; ++k) {
        const int64_t e = e0 + k * THREADS * 4;
        if (e >= 0 && e + 4 <= s.len) {
            const f32x4 x = load4<TYPE>(s.src, e);
            r.add(0, x.x);
            r.add(1, x.y);
            r.add(2, x.z);
            r.add(3, x.w);
        } else {
            for (int j = 0; j < 4; ++j)
                if (e + j >= 0 && e + j < s.len) r.add(j, load1<TYPE>(s.src, e + j));
        }
    }
}

template <int IN, int OUT, int THREADS>
__device__ __forceinline__ void clip_tile(const GradSeg &s, int64_t base, float f)
{
    constexpr int U = kGradTile / (THREADS * 4);
    const int64_t e0 = base + int(threadIdx.x) * 4;
    if (base >= 0 && base + kGradTile <= s.len) {
        f32x4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) x[k] = load4<IN>(s.src, e0 + k * THREADS * 4);
#pragma unroll
        for (int k = 0; k < U; ++k)
            store4<OUT>(s.dst, e0 + k * THREADS * 4,
                        f32x4{__fmul_rn(x[k].x, f), __fmul_rn(x[k].y, f), __fmul_rn(x[k].z, f), __fmul_rn(x[k].w, f)});
        return;
    }
    for (int k = 0; k < U; ++k) {
        const int64_t e = e0 + k * THREADS * 4;
        if (e >= 0 && e + 4 <= s.len) {
            const f32x4 x = load4<IN>(s.src, e);
            store4<OUT>(s.dst, e, f32x4{__fmul_rn(x.x, f), __fmul_rn(x.y, f), __fmul_rn(x.z, f), __fmul_rn(x.w, f)});
        } else {
            for (int j = 0; j < 4; ++j)
                if (e + j >= 0 && e + j < s.len) store1<OUT>(s.dst, e + j, __fmul_rn(load1<IN>(s.src, e + j), f));
        }
    }
}

template <int NORM, int THREADS>
__device__ __forceinline__ void norm_any(const GradTables &t, int tile, Running<NORM> &r)
{
    const GradSeg s = t.segs[t.tile_seg[tile]];
    const int64_t base = int64_t(tile - s.tile0) * kGradTile - s.shift;
    if (s.in == DDP_F32)
        norm_tile<NORM, DDP_F32, THREADS>(s, base, r);
    else if (s.in == DDP_BF16)
        norm_tile<NORM, DDP_BF16, THREADS>(s, base, r);
    else
        norm_tile<NORM, DDP_F16, THREADS>(s, base, r);
}

template <int IN, int THREADS>
__device__ __forceinline__ void clip_out(const GradSeg &s, int64_t base, float f)
{
    if (s.out == DDP_F32)
        clip_tile<IN, DDP_F32, THREADS>(s, base, f);
    else if (s.out == DDP_BF16)
        clip_tile<IN, DDP_BF16, THREADS>(s, base, f);
    else
        clip_tile<IN, DDP_F16, THREADS>(s, base, f);
}

// A factor of one leaves an in-place tensor as it is: x * 1 is x.
template <int THREADS>
__device__ __forceinline__ void clip_any(const GradTables &t, int tile, float f)
{
    const GradSeg s = t.segs[t.tile_seg[tile]];
    if (f == 1.0f && s.src == s.dst) return;
    const int64_t base = int64_t(tile - s.tile0) * kGradTile - s.shift;
    if (s.in == DDP_F32)
        clip_out<DDP_F32, THREADS>(s, base, f);
    else if (s.in == DDP_BF16)
        clip_out<DDP_BF16, THREADS>(s, base, f);
    else
        clip_out<DDP_F16, THREADS>(s, base, f);
}

constexpr int kNormThreads = 256;
constexpr int kSmallThreads = 1024;

template <int NORM>
__global__ void __launch_bounds__(kNormThreads) norm_partials(GradTables t, double *partials)
{
    Running<NORM> r;
    for (int tile = blockIdx.x; tile < t.norm_tiles; tile += gridDim.x) norm_any<NORM, kNormThreads>(t, tile, r);
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
        n = *(const GLOBAL float *)c.norm;
    } else {
        n = finished<NORM>(merged_partials<NORM, kNormThreads>(partials, n_partials));
        if (blockIdx.x == 0 && threadIdx.x == 0) *(GLOBAL float *)norm = n;
    }
    const float f = clip_factor(c.max_norm, n);
    // from the last tile down: the norm's pass left those in the caches
    for (int tile = t.all_tiles - 1 - int(blockIdx.x); tile >= 0; tile -= int(gridDim.x))
        clip_any<kNormThreads>(t, tile, f);
}

template <int NORM, bool CLIP>
__global__ void __launch_bounds__(kSmallThreads) small_list(GradTables t, float max_norm, float *norm)
{
    Running<NORM> r;
    for (int tile = 0; tile < t.norm_tiles; ++tile) norm_any<NORM, kSmallThreads>(t, tile, r);
    const float n = finished<NORM>(over_workgroup<NORM, kSmallThreads>(r.value()));
    if (threadIdx.x == 0) *(GLOBAL float *)norm = n;
    if (!CLIP) return;
    const float f = clip_factor(max_norm, n);
    for (int tile = 0; tile < t.all_tiles; ++tile) clip_any<kSmallThreads>(t, tile, f);
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
