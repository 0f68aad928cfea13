// Device helpers of the embedding kernels, shared by the translation units that
// instantiate them. Not part of the C ABI.
#pragma once

#include "../../include/ddp.h"
#include "embedding.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace ddp {
namespace {

#define GLOBAL __attribute__((address_space(1)))

// VEC elements of a type as they lie in memory, at any element's address.
template <int TYPE, int VEC>
struct Raw;
template <int VEC>
struct Raw<DDP_F32, VEC> {
    typedef float type __attribute__((ext_vector_type(VEC)));
    typedef type any __attribute__((aligned(4)));
    typedef float elem;
};
template <int VEC>
struct Raw<DDP_BF16, VEC> {
    typedef unsigned short type __attribute__((ext_vector_type(VEC)));
    typedef type any __attribute__((aligned(2)));
    typedef unsigned short elem;
};
template <int VEC>
struct Raw<DDP_F16, VEC> : Raw<DDP_BF16, VEC> {};

template <int TYPE, class E>
__device__ __forceinline__ float widen(E v)
{
    if constexpr (TYPE == DDP_F32)
        return v;
    else if constexpr (TYPE == DDP_BF16)
        return __uint_as_float(uint32_t(v) << 16);
    else
        return float(__builtin_bit_cast(_Float16, v));
}

// One rounding to the type, to nearest even; beyond fp16's range it is inf.
template <int TYPE>
__device__ __forceinline__ typename Raw<TYPE, 1>::elem narrow(float v)
{
    if constexpr (TYPE == DDP_F32) {
        return v;
    } else if constexpr (TYPE == DDP_BF16) {
        return __builtin_bit_cast(unsigned short, static_cast<__bf16>(v));
    } else {
        asm volatile("" : "+v"(v));   // an fp32 value before the conversion (see `wire` in reduce_kernels.h)
        return __builtin_bit_cast(unsigned short, static_cast<_Float16>(v));
    }
}

// STREAM: read past the caches.
template <int TYPE, int VEC, bool STREAM = false>
__device__ __forceinline__ typename Raw<TYPE, VEC>::type load(const void *base, int64_t e)
{
    const auto p = (const GLOBAL typename Raw<TYPE, VEC>::any *)(static_cast<const typename Raw<TYPE, VEC>::elem *>(base) + e);
    if constexpr (STREAM)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}

// Columns of a lane: VEC of them from `col` on. The last lane of a row whose
// width is no multiple of VEC loads the row's last VEC columns instead, which
// overlap its neighbour's, and stores only its own: `skip` of them are the
// neighbour's. Rows narrower than VEC go one column a lane (VEC = 1).
template <int VEC>
struct Columns {
    int64_t col;
    int skip;
    bool on;
    __device__ __forceinline__ Columns(int64_t slab, int lane, int64_t width)
    {
        const int64_t c = (slab * 64 + lane) * VEC;
        on = c < width;
        col = c + VEC <= width ? c : width - VEC;
        skip = int(c - col);
        if (!on) col = 0, skip = 0;   // loads of an idle lane stay inside the row
    }
};

// STREAM: written past the caches, which then keep what is read (rows of the
// table, of the gradient): lookup of 32767 rows of 2048 fp32 values into bf16
// 26.0 us against 40.4 with plain stores, gradient of 8191 positions of 2047
// written whole 30.4 against 39.8.
template <int TYPE, int VEC, bool STREAM = true>
__device__ __forceinline__ void store(void *base, int64_t e, const float (&v)[VEC], int skip)
{
    typedef Raw<TYPE, VEC> R;
    typename R::elem *p = static_cast<typename R::elem *>(base) + e;
    if (skip == 0) {
        typename R::type x;
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = narrow<TYPE>(v[j]);
        if constexpr (STREAM)
            __builtin_nontemporal_store(x, (GLOBAL typename R::any *)p);
        else
            *(GLOBAL typename R::any *)p = x;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (j >= skip) *(GLOBAL typename R::elem *)(p + j) = narrow<TYPE>(v[j]);
    }
}

// Data that no wave of the launch writes: uniform loads of it go through the
// scalar cache.
#define CONSTANT __attribute__((address_space(4)))

// The row of a token, or -1.
__device__ __forceinline__ int row_of(const EmbeddingArgs &a, int64_t tok)
{
    // unsigned, so that no index wraps into the range
    const uint64_t r = uint64_t(tok) - uint64_t(a.first_row);
    return r < uint64_t(a.n_rows) ? int(r) : -1;
}

// Waves of a launch that covers rows of any number, at most; further rows go to
// the next launch.
constexpr int64_t kMostWaves = int64_t(1) << 20;

constexpr int kWaves = 4;   // of a workgroup of the row kernels

__device__ __forceinline__ int wave_of()
{
    return __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 64);
}

// A workgroup's range of rows, as tests of a token: its row is below the range,
// or in it (at `local`). Every workgroup puts every token to both tests, so
// they are what the kernel spends its time on: two subtractions and two
// comparisons a token, the rest on the scalar unit.
struct Range {
    uint64_t first, lo, hi;
    __device__ __forceinline__ uint64_t row(int64_t tok) const { return uint64_t(tok) - first; }
    __device__ __forceinline__ bool below(uint64_t r) const { return r < lo; }
    __device__ __forceinline__ bool upto(uint64_t r) const { return r < hi; }
};

template <int GRAD, int VEC, bool ACC>
__device__ __forceinline__ void put(const EmbeddingArgs &a, void *grad, int row, const Columns<VEC> &c,
                                    const typename Raw<GRAD, VEC>::type &old, const float (&sum)[VEC])
{
    if (!c.on) return;
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        v[j] = ACC ? __fmaf_rn(a.scale, sum[j], widen<GRAD>(old[j])) : __fmul_rn(a.scale, sum[j]);
    store<GRAD, VEC>(grad, row * a.grad_stride + c.col, v, c.skip);
}

// A use of a loaded value that changes nothing: the compiler waits for the
// load here.
template <class T>
__device__ __forceinline__ void arrive(T &v)
{
    if constexpr (sizeof(T) >= 4) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 4); ++i) {
            uint32_t word;
            __builtin_memcpy(&word, reinterpret_cast<const char *>(&v) + 4 * i, 4);
            asm volatile("" : "+v"(word));
            __builtin_memcpy(reinterpret_cast<char *>(&v) + 4 * i, &word, 4);
        }
    } else {
        uint32_t word = v[0];
        asm volatile("" : "+v"(word));
        v[0] = static_cast<unsigned short>(word);
    }
}

template <int VEC>
int slabs_of(int64_t width)
{
    return int((width + 64 * VEC - 1) / (64 * VEC));
}

}  // namespace
}  // namespace ddp
