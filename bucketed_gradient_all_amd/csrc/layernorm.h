// Internal types shared by the host half of the layer norm (layernorm.cpp) and
// its kernels (layernorm.hip, layernorm_grad.hip). Not part of the C ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace ddp {

struct LayerArgs {
    int64_t rows, width;
    int64_t x_stride, add_stride, z_stride, y_stride;
    float eps;
    int32_t rms;      // no mean is taken off
    int32_t stream;   // the rows are read past the caches
    int32_t x_dtype, y_dtype, weight_dtype, grad_dtype;
};

// Columns of one load: 16 bytes of the wider type.
constexpr int layer_vector(int x_dtype, int y_dtype)
{
    return x_dtype == 0 || y_dtype == 0 ? 4 : 8;   // 0: DDP_F32
}

// Vectors of a row that the backward pass holds in registers, at most. Wider rows
// are read again for each pass over them.
constexpr int kRowVectors = 2048;

// The backward pass's workgroups, by the vectors of a row, their columns and
// whether rows are read past the caches: threads, and rows taken at once.
struct RowPlan {
    int threads, rows;
};
constexpr RowPlan row_plan(int64_t vectors, int64_t vec, bool stream)
{
    if (vectors > 512) return {512, 1};
    if (stream && vectors > 256 && vectors <= (vec == 4 ? 320 : 384)) return {192, 1};
    if (vectors > 256) return {512, 2};
    const int threads = stream ? 256 : 512;
    // three vectors a thread
    if (vectors > 64 && vectors <= 96 && stream) return {threads, threads / 32};
    if (vectors > 128 && vectors <= 192) return {threads, threads / 64};
    int shared = 8;   // threads of a row
    while (shared < vectors) shared *= 2;
    return {threads, threads / shared * 2};
}

struct LayerForward {
    const void *x, *add;   // add: or NULL
    const void *weight, *bias;   // or NULL
    void *z;                     // or NULL
    void *y;
    float *mean, *rstd;          // or NULL
};

struct LayerBackward {
    const void *dy, *z;
    const void *dz;              // or NULL
    const void *weight;          // or NULL
    const float *mean, *rstd;    // mean: NULL for DDP_RMS_NORM
    void *dx;                    // or NULL
    void *dweight, *dbias;       // or NULL
    float *parts;                // [n_parts][2][width] sums of dweight and dbias
    int32_t n_parts;             // workgroups that share the rows
    bool accumulate;
};

hipError_t launch_layernorm(const LayerArgs &a, const LayerForward &f, hipStream_t s);
// dx and the parts; rows that fit the registers.
hipError_t launch_layernorm_rows(const LayerArgs &a, const LayerBackward &b, hipStream_t s);
// All of a small call: dx, dweight and dbias; rows that fit the registers, and
// dx apart from dy.
hipError_t launch_layernorm_small(const LayerArgs &a, const LayerBackward &b, hipStream_t s);
// dx and the parts for rows of any width: the parts, then dx.
hipError_t launch_layernorm_wide(const LayerArgs &a, const LayerBackward &b, hipStream_t s);
// dweight and dbias from the parts.
hipError_t launch_layernorm_join(const LayerArgs &a, const LayerBackward &b, hipStream_t s);

}  // namespace ddp
