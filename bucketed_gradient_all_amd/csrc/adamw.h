// Internal types shared by the host half of the AdamW step (adamw.cpp) and its
// kernel (adamw.hip). Not part of the C ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace ddp {

// Elements of one tile: four a thread of a workgroup of 256. With eight workgroups
// a CU, and codes that went past the caches, 953M elements with a copy took 4.66 ms,
// against 4.87 with tiles of 2048 and 4.60 with tiles of 512 (128 threads); with
// 8-bit states 2.58, 2.70 and 2.60 ms, and 161 odd tensors of 25M elements 83, 87
// and 89 us. A list of eight tensors is a launch of 34 tiles (3.3 us in a graph;
// tiles of 2048 4.3).
constexpr int kAdamTile = 1024;

// Elements of the 8-bit states that share a scale.
constexpr int kStateBlock = 128;

// How a tensor's parameters are held: alone, or in fp32 with a 16-bit copy
// that is written beside them.
enum AdamOut : uint8_t { kParamF32, kParamF32CopyBF16, kParamF32CopyF16, kParamBF16, kParamF16 };

// One tensor. With 32-bit states its tiles are cut at parameter addresses that
// are multiples of 256 bytes, so that full tiles store whole cache lines: tile
// k covers elements [k * kAdamTile - shift, (k + 1) * kAdamTile - shift) of it.
// With 8-bit states shift is 0 and a tile holds eight whole blocks.
struct AdamSeg {
    const void *grad;
    void *param;
    void *copy;
    void *m, *v;               // fp32, or e4m3 codes
    float *m_scale, *v_scale;  // one a block, 8-bit states only
    int64_t len;
    double decay;
    int32_t tile0;   // first tile
    int16_t shift;   // 0..127
    uint8_t type;    // of the gradient: DDP_F32, DDP_BF16, DDP_F16
    AdamOut out;
};
static_assert(sizeof(AdamSeg) == 80, "tensor records are five 16-byte loads");

struct AdamTables {
    const AdamSeg *segs;
    const int32_t *tile_seg;   // tile -> tensor record
    int32_t tiles;
    int32_t bits;              // of the states: 32 or 8
};

struct AdamArgs {
    double lr, beta1, beta2;
    float b1, a1;   // beta1, 1 - beta1
    float b2, a2;
    float eps;
    float size;     // lr / (1 - beta1^t)
    float root;     // 1 / sqrt(1 - beta2^t)
    float max_norm;
    int64_t step;            // t
    const float *norm;       // or NULL
    const float *lr_ptr;     // or NULL: lr. Without both pointers size and root are set
    const int64_t *step_ptr; // or NULL: step
    int32_t skip;            // nothing is written if the norm is not finite
};

// b^t by squaring, for 0 <= b < 1 and t >= 0: the same bits on the host and on
// the device. Its relative error is at most about t * 2^-53, which the result's
// distance from 1 never shows in fp32: b^t itself vanishes long before. Below
// 2^-60 it is 0, its distance from 1 is 1 in 64 bits.
constexpr double power(double b, int64_t t)
{
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        if (r < 0x1p-60) return 0.0;
        b *= b;
    }
    return r;
}

hipError_t launch_adamw(const AdamTables &t, const AdamArgs &a, hipStream_t s);

}  // namespace ddp
