// Internal types shared by the host half of the embedding operators
// (embedding.cpp) and their kernels (embedding.hip). Not part of the C ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace ddp {

constexpr int kSortThreads = 1024;             // 16 waves
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxSortRows = 2048;             // rows of one sorting workgroup: 144 KiB of LDS counters

// Sorted positions one wave sums (a chunk), at most: it holds twice as many in
// its 64 lanes.
constexpr int kMaxChunk = 32;

// Columns a lane sums: 16 bytes of the wider type.
constexpr int sum_vector(int act_dtype, int grad_dtype)
{
    return act_dtype == 0 || grad_dtype == 0 ? 4 : 8;   // 0: DDP_F32
}

struct EmbeddingArgs {
    int64_t n_rows, width;
    int64_t first_row;
    int64_t table_stride, grad_stride, act_stride;
    int64_t n_tokens;
    float scale;
    int32_t index64;
    int32_t table_dtype, grad_dtype, act_dtype;
};

// The gradient's workspace.
struct EmbeddingWork {
    int32_t *row;     // [T] rows of the sorted positions
    int32_t *pos;     // [T] the positions, sorted by row, then by position
    int32_t *begin;   // [V + 1] where each row's positions begin; the last: how many lie in the table
    float *first;     // [chunks][slots] sums of the pieces that begin a long run
    float *more;      // [chunks][slots] sums of the pieces that go on with one
    int64_t pitch;    // elements of one chunk's slot: the width rounded up
    int32_t chunk;    // positions of a chunk
    int32_t n_chunks;
    int32_t sort_rows;   // rows of one sorting workgroup
    int32_t splits;      // sorting workgroups of one range of rows
    int32_t stream;      // read dout past the caches
    int32_t pad_row;     // the row whose positions count for nothing, or -1
};

// A small batch's gradient in one launch: positions it takes at most (an entry
// holds a position in 16 bits, a wave four groups of 64 tokens), and rows of a
// workgroup's range (one a thread).
constexpr int kSmallTokens = 4096, kSmallRows = 1024;

struct SmallPlan {
    int32_t rows;      // of a workgroup's range
    int32_t slabs;     // of columns
    int32_t pad_row;   // the row whose positions count for nothing, or -1
};

hipError_t launch_small_grad(const EmbeddingArgs &a, const SmallPlan &p, const void *tokens, const void *dout,
                             void *grad, bool accumulate, hipStream_t s);
hipError_t launch_lookup(const EmbeddingArgs &a, const void *table, const void *tokens, void *out, hipStream_t s);
hipError_t launch_sort(const EmbeddingArgs &a, const void *tokens, const EmbeddingWork &w, hipStream_t s);
hipError_t launch_sum(const EmbeddingArgs &a, const void *dout, void *grad, bool accumulate, const EmbeddingWork &w,
                      hipStream_t s);
hipError_t launch_join(const EmbeddingArgs &a, void *grad, bool accumulate, const EmbeddingWork &w, hipStream_t s);

}  // namespace ddp
