// Device helpers of the layer norm's kernels. Not part of the C ABI.
#pragma once

#include "../../include/ddp.h"
#include "element.h"
#include "layernorm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

namespace ddp {
namespace {

// VEC columns of a row from `col` on, of which the first `skip` belong to the
// vector before: the last vector of a row whose width is no multiple of VEC
// takes the row's last VEC columns. VEC of them are skipped past the row.
template <int VEC>
struct Columns {
    int64_t col;
    int skip;
    __device__ __forceinline__ Columns(int64_t vector, int64_t width)
    {
        const int64_t c = vector * VEC;
        const bool on = c < width;
        col = !on ? 0 : c + VEC <= width ? c : width - VEC;   // an idle thread's loads stay inside the row
        skip = on ? int(c - col) : VEC;
    }
};

// STREAM: past the caches.
template <int TYPE, int VEC, bool STREAM = false>
__device__ __forceinline__ typename Raw<TYPE, VEC>::type load(const void *base, int64_t e)
{
    const auto p = (const GLOBAL typename Raw<TYPE, VEC>::any *)(static_cast<const typename Raw<TYPE, VEC>::elem *>(base) + e);
    if constexpr (STREAM)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}

template <int TYPE>
__device__ __forceinline__ const void *row_of(const void *p, int64_t row, int64_t stride)
{
    return static_cast<const typename Raw<TYPE, 1>::elem *>(p) + row * stride;
}

template <int TYPE>
__device__ __forceinline__ void *row_of(void *p, int64_t row, int64_t stride)
{
    return static_cast<typename Raw<TYPE, 1>::elem *>(p) + row * stride;
}

template <int TYPE, int VEC>
__device__ __forceinline__ void widen_all(const typename Raw<TYPE, VEC>::type &x, float (&v)[VEC])
{
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = widen<TYPE>(x[j]);
}

// Written past the caches: 32768 rows of 2048 bf16 values forward 94 us against
// 102, 16384 of 1024 fp32 values 54 against 58; with a kernel behind it that reads
// y, 2048 rows of 2048 10.9 against 12.3, 8192 rows 36.8 against 34.4.
template <int TYPE, int VEC>
__device__ __forceinline__ void store(void *base, int64_t e, const float (&v)[VEC], int skip)
{
    typedef Raw<TYPE, VEC> R;
    typename R::elem *p = static_cast<typename R::elem *>(base) + e;
    typename R::type x;
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = narrow<TYPE>(v[j]);
    if (skip == 0) {
        __builtin_nontemporal_store(x, (GLOBAL typename R::any *)p);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (j >= skip) *(GLOBAL typename R::elem *)(p + j) = x[j];
    }
}

// Columns of weight or bias, or `otherwise` without one.
template <int VEC>
__device__ __forceinline__ void load_weight(const void *w, int type, int64_t col, float otherwise, float (&v)[VEC])
{
    if (!w) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = otherwise;
    } else if (type == DDP_F32) {
        widen_all<DDP_F32, VEC>(load<DDP_F32, VEC>(w, col), v);
    } else if (type == DDP_BF16) {
        widen_all<DDP_BF16, VEC>(load<DDP_BF16, VEC>(w, col), v);
    } else {
        widen_all<DDP_F16, VEC>(load<DDP_F16, VEC>(w, col), v);
    }
}

template <int CONTROL>
__device__ __forceinline__ float with_lane(float x)
{
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CONTROL, 0xf, 0xf, false));
}

// The sum over the sixteens that T lanes are, lane by lane, in each of them.
template <int T>
__device__ __forceinline__ float across_rows(float x)
{
    if (T >= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    if (T >= 64) {
        const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(b[0]) + __uint_as_float(b[1]);
    }
    return x;
}

// The sum of T neighbouring lanes' values, the same bits in each of them.
template <int T>
__device__ __forceinline__ float lane_sum(float x)
{
    x = with_lane<0xb1>(x);    // the neighbour
    x = with_lane<0x4e>(x);    // the other pair of four
    x = with_lane<0x141>(x);   // the other four of eight
    if (T >= 16) x = with_lane<0x140>(x);   // the other eight of sixteen
    return across_rows<T>(x);
}

// Which of the workgroup's rows a thread works on, where T threads share one.
template <int T>
__device__ __forceinline__ int group_of()
{
    const int group = int(threadIdx.x) / T;
    return T >= 64 ? __builtin_amdgcn_readfirstlane(group) : group;
}

// Sums over the T threads that share a row, the same bits in each of them: lanes
// of a wave, or several waves of a workgroup of THREADS, whose threads call it
// together then; `turn` counts the calls, so that one barrier a call is enough.
template <int T, int THREADS, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int &turn)
{
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lane_sum<T>(v[k]);
    if constexpr (T > 64) {
        __shared__ float part[2][THREADS / 64][N];
        constexpr int WAVES = T / 64;
        const int wave = int(threadIdx.x) / 64, slot = turn & 1;
        const int first = THREADS == T ? 0 : wave / WAVES * WAVES;
        ++turn;
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) part[slot][wave][k] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = part[slot][first][k];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v[k] += part[slot][first + w][k];
        }
    }
}

// Workgroups of one launch: its grid holds 2^32 threads.
constexpr int64_t kMostGroups = int64_t(1) << 21;

// f(x type, y type) for the pairs that a desc may hold.
template <class F>
hipError_t by_types(const LayerArgs &a, F &&f)
{
    using std::integral_constant;
    typedef integral_constant<int, DDP_F32> F32;
    typedef integral_constant<int, DDP_BF16> BF16;
    typedef integral_constant<int, DDP_F16> F16;
    if (a.x_dtype == DDP_BF16) return f(BF16(), BF16());
    if (a.x_dtype == DDP_F16) return f(F16(), F16());
    if (a.y_dtype == DDP_BF16) return f(F32(), BF16());
    if (a.y_dtype == DDP_F16) return f(F32(), F16());
    return f(F32(), F32());
}

}  // namespace
}  // namespace ddp
