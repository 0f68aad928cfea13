// Internal types shared by the host half of the gradient lists
// (grad_list.cpp) and their kernels (grad_norm.hip). Not part of the C ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace ddp {

// Elements of one tile. A workgroup of 256 threads takes a tile in eight
// groups of four elements a thread: 32 KiB of fp32 in flight a workgroup.
constexpr int kGradTile = 8192;

// Lists of up to this many tiles are handled by one workgroup in one launch:
// the norm, and the norm with clipping. Replayed from a graph, one launch
// against two, the tiles full: the norm of 4 tiles 3.3 us against 4.7, of 12
// 5.4 against 4.9; clipping of 4 tiles into another buffer 5.8 against 5.6, of
// 12 12.3 against 5.7. Called one by one, the second launch costs the host
// about 3 us more.
constexpr int kSmallNorm = 12, kSmallClip = 6;

// Most workgroups the norm's pass is split over: each leaves one 8-byte
// partial, and the last step sums them in index order.
constexpr int kMaxPartials = 1024;

// Lists of more than this many tiles that are clipped into other buffers are
// clipped by a workgroup a part of a tile, with the norm finished by a launch
// of its own before. That launch takes 4 to 5 us, the parts are a few percent
// faster: replayed from a graph, fp32 into fp32, 2048 tiles 38.6 us against
// 37.9 with workgroups that go from tile to tile, 4096 70.3 against 69.3, 8192
// 133 against 136, 65536 1056 against 1126; bf16 into fp32, 1024 18.2 against
// 18.1, 4096 49.1 against 50.2, 65536 691 against 752.
constexpr int kManyTiles = 4096;

// One tensor of a list. Its tiles are cut at absolute destination addresses
// that are multiples of 256 bytes, whatever address the tensor starts at, so
// that full tiles store whole cache lines: tile k of the tensor covers
// elements [k * kGradTile - shift, (k + 1) * kGradTile - shift) of it.
struct GradSeg {
    const void *src;
    void *dst;
    int64_t len;
    int32_t tile0;   // first tile
    int16_t shift;   // 0..127
    uint8_t in;      // DDP_F32, DDP_BF16, DDP_F16
    uint8_t out;
};
static_assert(sizeof(GradSeg) == 32, "tensor records are two 16-byte loads");

struct GradTables {
    const GradSeg *segs;
    const int32_t *tile_seg;   // tile -> tensor record
    int32_t norm_tiles;        // the first copy's tiles: what the norm is taken over
    int32_t all_tiles;         // every copy's: what clipping scales
    int32_t in_place;          // clipping writes where it reads
};

// Where clipping takes the norm from.
struct ClipFactor {
    float max_norm;
    const float *norm;   // given norm, or NULL: reduce the partials
};

// norm_type: DDP_NORM_*. blocks: workgroups (and partials) of the pass over
// the gradients, a rule of the host.
hipError_t launch_norm_partials(int norm_type, const GradTables &t, int blocks, void *partials, hipStream_t s);
hipError_t launch_norm_finish(int norm_type, int blocks, const void *partials, float *norm, hipStream_t s);
// Scales every copy; with f.norm NULL the norm comes from the partials, and
// the first workgroup writes it to `norm`.
hipError_t launch_clip(int norm_type, const GradTables &t, int blocks, const ClipFactor &f, int n_partials,
                       const void *partials, float *norm, hipStream_t s);
hipError_t launch_clip_parts(const GradTables &t, const ClipFactor &f, hipStream_t s);
// One workgroup: the norm, and with clip != 0 the scaling too.
hipError_t launch_small(int norm_type, const GradTables &t, bool clip, float max_norm, float *norm, hipStream_t s);

}  // namespace ddp
