// One AdamW step over a list of tensors.
//
//   g = grad * f,  f = min(1, max_norm / (norm + 1e-6)), or 1 without a norm
//   m = beta1 * m + (1 - beta1) * g
//   v = beta2 * v + (1 - beta2) * g^2
//   p = p * (1 - lr * decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//   copy = R(p)                                  R: one rounding to the copy's type
//
// One pass over memory and no operand used twice, so it is bound by memory: 335M
// fp32 parameters 1.55 ms (6.1 TB/s), 953M with bf16 gradients and a bf16 copy
// 4.4 ms (6.1 TB/s), with 8-bit states 2.49 ms (6.2 TB/s). Everything is fp32 and
// every operation is rounded by itself (no product is fused with a sum). The
// root and the quotient are IEEE's over fp32's whole range, but for the quotient of
// the 8-bit step (below): an element takes some seventy-five instructions there,
// close to what the memory's time leaves.
//
// 8-bit states: the m and r = sqrt(v) of a block of 128 elements are held as
// e4m3 codes of m * (1 / max|m| * 448), with max|m| * (1 / 448) as the block's scale.
//   * The root, because the codes' range of 2^-9 to 448 then spans 2^35 of v, and
//     because the root is what the step divides by.
//   * A positive r never gets the code of zero: with r = 0 beside an m that is
//     not, a later step with a small gradient would divide by eps alone. A root
//     that is held too large only makes that element's step smaller.
//   * The step itself uses this step's m and v before they are rounded.
//   * The maximum is taken on the bit patterns as unsigned integers, where an
//     infinity and a NaN are above every number: the scale is then not finite
//     either, and no state of the block is.
#include "../../include/ddp.h"
#include "adamw.h"
#include "element.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>

namespace ddp {
namespace {

constexpr int kVec = 4;
constexpr int kThreads = 256;
static_assert(kAdamTile == kThreads * kVec, "one vector a thread");

template <int TYPE>
using Vec = typename Raw<TYPE, kVec>::type;

// Those of four elements that the tensor has.
struct Some {
    int lo, hi;
    __device__ __forceinline__ bool all() const { return lo == 0 && hi == kVec; }
};

template <bool FULL>
__device__ __forceinline__ Some some_of(int64_t e, int64_t len)
{
    if (FULL) return {0, kVec};
    return {int(min(int64_t(kVec), max(int64_t(0), -e))), int(max(int64_t(0), min(int64_t(kVec), len - e)))};
}

template <int TYPE>
__device__ __forceinline__ Vec<TYPE> load(const void *base, int64_t e, Some n)
{
    typedef Raw<TYPE, kVec> R;
    const GLOBAL typename R::elem *p = (const GLOBAL typename R::elem *)base + e;
    if (n.all()) return __builtin_nontemporal_load((const GLOBAL typename R::any *)p);
    Vec<TYPE> x = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (j >= n.lo && j < n.hi) x[j] = p[j];
    return x;
}

template <int TYPE>
__device__ __forceinline__ void store(void *base, int64_t e, Some n, const float (&v)[kVec])
{
    typedef Raw<TYPE, kVec> R;
    GLOBAL typename R::elem *p = (GLOBAL typename R::elem *)base + e;
    Vec<TYPE> x;
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = narrow<TYPE>(v[j]);
    if (n.all()) {
        __builtin_nontemporal_store(x, (GLOBAL typename R::any *)p);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j >= n.lo && j < n.hi) p[j] = x[j];
    }
}

// What a step multiplies with, the same for a tensor's elements.
struct Scalars {
    float f, b1, a1, b2, a2, eps, size, root;
    float keep;   // 1 - lr * decay
};

// False: the step is left out.
__device__ __forceinline__ bool scalars_of(const AdamArgs &a, double decay, Scalars *c)
{
    *c = {1.0f, a.b1, a.a1, a.b2, a.a2, a.eps, a.size, a.root, 1.0f};
    double lr = a.lr;
    if (a.norm) {
        const float n = *(const CONSTANT float *)a.norm;
        if (a.skip && !(fabsf(n) < INFINITY)) return false;
        if (a.max_norm < INFINITY) c->f = clip_factor(a.max_norm, n);
    }
    if (a.lr_ptr || a.step_ptr) {
        // one wave's 64-bit powers for the workgroup: 42M elements with 8-bit
        // states 94 to 98 us at step 2000, 86 with the host's scalars; 953M 2.55
        // ms and 2.48 (all four waves' powers took a quarter and a tenth more)
        __shared__ float found[2];
        if (a.lr_ptr) lr = double(*(const CONSTANT float *)a.lr_ptr);
        if (threadIdx.x < 64) {
            const int64_t t = a.step_ptr ? max(int64_t(1), *(const CONSTANT int64_t *)a.step_ptr) : a.step;
            const float size = float(lr / (1.0 - power(a.beta1, t)));
            const float root = float(1.0 / __builtin_sqrt(1.0 - power(a.beta2, t)));
            if (threadIdx.x == 0) found[0] = size, found[1] = root;
        }
        __syncthreads();
        c->size = found[0];
        c->root = found[1];
    }
    c->keep = float(1.0 - lr * decay);
    return true;
}

// a / b for b in [0, 2^126]: the remainder of a first quotient corrects it once, to
// nearest, or beside it where a / b lies all but in the middle of two values (it
// equals IEEE division for every reciprocal and for 2^31 random quotients). Where
// the remainder is subnormal (|a| below 2^-100) the quotient is off by two units in
// its last place at most. A first quotient beyond fp32's range is held at its end,
// from where the correction leaves it where it belongs. IEEE division, scaled and
// corrected twice, takes four instructions more: 42M elements with 8-bit states 90
// us against 87.5, with the schedule on the device 101 against 98, 953M 2.62 ms
// against 2.55; with 32-bit states it is free.
__device__ __forceinline__ float quotient(float a, float b)
{
    float r = __builtin_amdgcn_rcpf(b);
    r = __fmaf_rn(__fmaf_rn(-b, r, 1.0f), r, r);
    float q = __builtin_amdgcn_fmed3f(a * r, -FLT_MAX, FLT_MAX);
    q = __fmaf_rn(__fmaf_rn(-b, q, a), r, q);
    return __builtin_amdgcn_div_fixupf(q, b, a);   // zeros, infinities and NaN
}

// One element's step; returns sqrt(v).
template <int BITS>
__device__ __forceinline__ float update(const Scalars &c, float g, float &m, float &v, float &p)
{
    g = __fmul_rn(g, c.f);
    m = __fadd_rn(__fmul_rn(m, c.b1), __fmul_rn(g, c.a1));
    v = __fadd_rn(__fmul_rn(v, c.b2), __fmul_rn(__fmul_rn(g, g), c.a2));
    const float r = sqrtf(v);   // to nearest, for a subnormal v too
    const float b = __fadd_rn(__fmul_rn(r, c.root), c.eps);
    const float d = BITS == 32 ? __fdiv_rn(m, b) : quotient(m, b);
    p = __fsub_rn(__fmul_rn(p, c.keep), __fmul_rn(d, c.size));
    return r;
}

template <AdamOut OUT>
struct Types {
    static constexpr int param = OUT == kParamBF16 ? DDP_BF16 : OUT == kParamF16 ? DDP_F16 : DDP_F32;
    static constexpr int copy = OUT == kParamF32CopyBF16 ? DDP_BF16 : OUT == kParamF32CopyF16 ? DDP_F16 : -1;
};

template <int GRAD, AdamOut OUT, bool FULL>
__device__ __forceinline__ void step_32(const CONSTANT AdamSeg &s, int64_t base, const AdamArgs &a)
{
    typedef Types<OUT> T;
    const int64_t e = base + int(threadIdx.x) * kVec;
    const Some n = some_of<FULL>(e, s.len);
    const Vec<GRAD> g = load<GRAD>(s.grad, e, n);
    const Vec<T::param> p = load<T::param>(s.param, e, n);
    const Vec<DDP_F32> m = load<DDP_F32>(s.m, e, n), v = load<DDP_F32>(s.v, e, n);
    Scalars c;
    if (!scalars_of(a, s.decay, &c)) return;   // behind the loads: it takes a load and a division of its own
    float x[kVec], y[kVec], z[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        x[j] = widen<T::param>(p[j]), y[j] = m[j], z[j] = v[j];
        update<32>(c, widen<GRAD>(g[j]), y[j], z[j], x[j]);
    }
    store<T::param>(s.param, e, n, x);
    if constexpr (T::copy >= 0) store<T::copy>(s.copy, e, n, x);
    store<DDP_F32>(s.m, e, n, y);
    store<DDP_F32>(s.v, e, n, z);
}

typedef uint32_t codes_any __attribute__((aligned(1)));

// The codes of four elements, those the tensor has not as zeros. Codes go through
// the caches: a wave's are two cache lines, of which tensors that do not begin at
// one fill only parts, which the cache joins (161 odd tensors 72 us against 82
// past the caches). Everything else goes past them: 1.56 ms against 1.73 for the
// 335M fp32 elements.
__device__ __forceinline__ uint32_t load_codes(const void *base, int64_t e, Some n)
{
    const GLOBAL uint8_t *p = (const GLOBAL uint8_t *)base + e;
    if (n.all()) return *(const GLOBAL codes_any *)p;
    uint32_t x = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (j >= n.lo && j < n.hi) x |= uint32_t(p[j]) << (8 * j);
    return x;
}

__device__ __forceinline__ void store_codes(void *base, int64_t e, Some n, uint32_t x)
{
    GLOBAL uint8_t *p = (GLOBAL uint8_t *)base + e;
    if (n.all()) {
        *(GLOBAL codes_any *)p = x;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j >= n.lo && j < n.hi) p[j] = uint8_t(x >> (8 * j));
    }
}

__device__ __forceinline__ void decode(uint32_t code, float scale, float (&x)[kVec])
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(code), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(code), true);
    x[0] = __fmul_rn(lo[0], scale), x[1] = __fmul_rn(lo[1], scale);
    x[2] = __fmul_rn(hi[0], scale), x[3] = __fmul_rn(hi[1], scale);
}

__device__ __forceinline__ uint32_t encode(const float (&x)[kVec])
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true));
}

template <int CONTROL>
__device__ __forceinline__ uint32_t max_with(uint32_t x)
{
    return max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CONTROL, 0xf, 0xf, false)));
}

// The largest of a half wave's values, in each of its lanes.
__device__ __forceinline__ uint32_t over_half_wave(uint32_t x)
{
    x = max_with<0xb1>(x);    // the neighbour
    x = max_with<0x4e>(x);    // the other pair of four
    x = max_with<0x141>(x);   // the other four of eight
    x = max_with<0x140>(x);   // the other eight of sixteen
    const auto y = __builtin_amdgcn_permlane16_swap(x, x, false, false);   // the other sixteen of thirty-two
    return max(uint32_t(y[0]), uint32_t(y[1]));
}

// x of the even or the odd lane of each pair.
template <int ODD>
__device__ __forceinline__ float of_pair(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ODD ? 0xf5 : 0xa0, 0xf, 0xf, false));
}

// Of a block's largest magnitude: what its values are multiplied with before
// they are rounded to codes, and the scale that undoes it. A block whose
// largest is below 2^-100, where 1 / top * 448 could overflow, is held as zeros.
// top is divided by 256 before and 448 after, both exactly: the reciprocal is then
// normal up to fp32's end (beyond 2^126 it is not rounded to a subnormal number).
struct BlockScale {
    float up, down;
    __device__ __forceinline__ explicit BlockScale(uint32_t top_bits)
    {
        const float top = __uint_as_float(top_bits);
        const bool none = top < 0x1p-100f;
        up = none ? 0.0f : __fmul_rn(quotient(1.0f, top * 0x1p-8f), 448.0f * 0x1p-8f);
        down = none ? 0.0f : __fmul_rn(top, 1.0f / 448.0f);
    }
};

// A block lies in half a wave, so that every load and store is one range of whole
// cache lines a wave. (Blocks in sixteen lanes, two vectors each, need a tenth
// fewer instructions, but store codes in pieces of 64 bytes: the 1B decoder's
// step 2.75 ms against 2.50.) Even lanes compute the first moment's scales, odd
// ones the second's.
static_assert(kStateBlock == 32 * kVec, "half a wave");

template <int GRAD, AdamOut OUT, bool FULL>
__device__ __forceinline__ void step_8(const CONSTANT AdamSeg &s, int64_t base, const AdamArgs &a)
{
    typedef Types<OUT> T;
    const int64_t e = base + int(threadIdx.x) * kVec;
    const Some n = some_of<FULL>(e, s.len);
    const int64_t block = e >> 7;
    const bool has = FULL || block << 7 < s.len;   // a block that begins inside the tensor has a scale
    const float ms = has ? ((const GLOBAL float *)s.m_scale)[block] : 0.0f;
    const float vs = has ? ((const GLOBAL float *)s.v_scale)[block] : 0.0f;
    const uint32_t m = load_codes(s.m, e, n), v = load_codes(s.v, e, n);
    const Vec<GRAD> g = load<GRAD>(s.grad, e, n);
    const Vec<T::param> p = load<T::param>(s.param, e, n);
    Scalars c;
    if (!scalars_of(a, s.decay, &c)) return;   // behind the loads: it takes a load and a division of its own
    float x[kVec], y[kVec], r[kVec];
    decode(m, ms, y);
    decode(v, vs, r);
    uint32_t top_m = 0, top_r = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        x[j] = widen<T::param>(p[j]);
        float z = __fmul_rn(r[j], r[j]);
        r[j] = update<8>(c, widen<GRAD>(g[j]), y[j], z, x[j]);
        top_m = max(top_m, __float_as_uint(y[j]) & 0x7fffffffu);
        top_r = max(top_r, __float_as_uint(r[j]));   // not negative; a NaN of either sign is above all
    }
    store<T::param>(s.param, e, n, x);
    if constexpr (T::copy >= 0) store<T::copy>(s.copy, e, n, x);
    top_m = over_half_wave(top_m);
    top_r = over_half_wave(top_r);
    const bool odd = threadIdx.x & 1;
    const BlockScale b(odd ? top_r : top_m);
    const float up_m = of_pair<0>(b.up), up_r = of_pair<1>(b.up);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        y[j] = __fmul_rn(y[j], up_m);
        // 2^-9 is the smallest code
        r[j] = r[j] > 0.0f ? fmaxf(__fmul_rn(r[j], up_r), 0x1p-9f) : 0.0f;
    }
    store_codes(s.m, e, n, encode(y));
    store_codes(s.v, e, n, encode(r));
    if ((threadIdx.x & 30) == 0 && has) ((GLOBAL float *)(odd ? s.v_scale : s.m_scale))[block] = b.down;
}

template <int BITS, int GRAD, AdamOut OUT>
__device__ __forceinline__ void step_tile(const CONSTANT AdamSeg &s, int64_t base, const AdamArgs &a)
{
    const bool full = base >= 0 && base + kAdamTile <= s.len;
    if (BITS == 32) {
        if (full)
            step_32<GRAD, OUT, true>(s, base, a);
        else
            step_32<GRAD, OUT, false>(s, base, a);
    } else {
        if (full)
            step_8<GRAD, OUT, true>(s, base, a);
        else
            step_8<GRAD, OUT, false>(s, base, a);
    }
}

template <int BITS, int GRAD>
__device__ __forceinline__ void step_out(const CONSTANT AdamSeg &s, int64_t base, const AdamArgs &a)
{
    switch (s.out) {
    case kParamF32: step_tile<BITS, GRAD, kParamF32>(s, base, a); break;
    case kParamF32CopyBF16: step_tile<BITS, GRAD, kParamF32CopyBF16>(s, base, a); break;
    case kParamF32CopyF16: step_tile<BITS, GRAD, kParamF32CopyF16>(s, base, a); break;
    case kParamBF16: step_tile<BITS, GRAD, kParamBF16>(s, base, a); break;
    default: step_tile<BITS, GRAD, kParamF16>(s, base, a); break;
    }
}

template <int BITS>
__global__ void __launch_bounds__(kThreads) adamw(AdamTables t, AdamArgs a, int first)
{
    const int tile = first + int(blockIdx.x);
    const CONSTANT AdamSeg &s = ((const CONSTANT AdamSeg *)t.segs)[((const CONSTANT int32_t *)t.tile_seg)[tile]];
    const int64_t base = int64_t(tile - s.tile0) * kAdamTile - s.shift;
    if (s.type == DDP_F32)
        step_out<BITS, DDP_F32>(s, base, a);
    else if (s.type == DDP_BF16)
        step_out<BITS, DDP_BF16>(s, base, a);
    else
        step_out<BITS, DDP_F16>(s, base, a);
}

// Tiles of one launch: its grid holds 2^32 threads.
constexpr int32_t kMostTiles = int32_t(1) << 23;

// LDS that a workgroup of the 32-bit step reserves and does not use, so that four
// fit a CU: fewer streams at once suit the memory. 335M elements take 1.52 ms
// with four a CU, 1.58 with three, 1.57 with five, 1.62 with eight; 953M with a
// copy 4.33, 4.40, 4.46 and 4.66. The 8-bit step has more to compute for each
// byte and takes all eight (2.48 ms; four 3.17, six 2.59).
constexpr unsigned kReserved = 40000;

}  // namespace

hipError_t launch_adamw(const AdamTables &t, const AdamArgs &a, hipStream_t s)
{
    for (int32_t first = 0; first < t.tiles; first += kMostTiles) {
        const dim3 g(static_cast<unsigned>(std::min(kMostTiles, t.tiles - first)));
        if (t.bits == 32)
            hipLaunchKernelGGL(adamw<32>, g, dim3(kThreads), kReserved, s, t, a, first);
        else
            hipLaunchKernelGGL(adamw<8>, g, dim3(kThreads), 0, s, t, a, first);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace ddp
