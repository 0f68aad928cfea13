// Elements of the three types as the kernels read and write them: vectors at
// any element's address, widening to fp32 and one rounding back. Not part of
// the C ABI.
#pragma once

#include "../../include/ddp.h"

#include <hip/hip_runtime.h>

namespace ddp {
namespace {

#define GLOBAL __attribute__((address_space(1)))
// Data that no wave of the launch writes: uniform loads of it go through the
// scalar cache.
#define CONSTANT __attribute__((address_space(4)))

// VEC elements as they lie in memory, at any element's address: tensors start
// where they do, and global memory takes vectors at any address.
template <int TYPE, int VEC>
struct Raw;
template <int VEC>
struct Raw<DDP_F32, VEC> {
    typedef float elem;
    typedef float type __attribute__((ext_vector_type(VEC)));
    typedef type any __attribute__((aligned(4)));
};
template <int VEC>
struct Raw<DDP_BF16, VEC> {
    typedef unsigned short elem;
    typedef unsigned short type __attribute__((ext_vector_type(VEC)));
    typedef type any __attribute__((aligned(2)));
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
        // an fp32 value, rounded by itself, before the conversion (see `wire`
        // in reduce_kernels.h)
        asm volatile("" : "+v"(v));
        return __builtin_bit_cast(unsigned short, static_cast<_Float16>(v));
    }
}

// What gradients are scaled by, wherever they are clipped. A NaN stays one.
__device__ __forceinline__ float clip_factor(float max_norm, float norm)
{
    const float f = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
    return f >= 1.0f ? 1.0f : f;
}

}  // namespace
}  // namespace ddp
