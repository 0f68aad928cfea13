// Error recording and the exception guard of the C ABI's entry points, shared
// by the host sources. Not part of the C ABI.
#pragma once

#include "../../include/ddp.h"

#include <hip/hip_runtime_api.h>

#include <new>
#include <string>

namespace ddp {

// Record the thread's last error text (ddp_last_error) and return the code.
// Recording never throws. Defined in reducer.cpp.
int fail(int code, const std::string &msg) noexcept;
int fail(int code, const char *msg) noexcept;
int hip_fail(const char *what, hipError_t e) noexcept;
int no_memory() noexcept;

// Every entry point runs its body through this: the C ABI never lets an
// exception out. Host memory exhaustion (std::bad_alloc from a container or
// a message) becomes DDP_ERR_NOMEM; anything else DDP_ERR_INVALID.
template <class F>
int guarded(F &&body) noexcept
{
    try {
        return body();
    } catch (const std::bad_alloc &) {
        return no_memory();
    } catch (...) {
        return fail(DDP_ERR_INVALID, "internal error: unexpected exception in the host library");
    }
}

// The stream of a call. hipStreamLegacy is another name of the null stream.
inline hipStream_t stream_of(void *stream) noexcept
{
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return s == hipStreamLegacy ? nullptr : s;
}

// DDP_OK if work on stream s runs on `device`, the current one. Defined in
// grad_list.cpp.
int check_stream(hipStream_t s, int device);

// What a reducer's gradient list is made of (ddp_grads_from_reducer).
// Defined in reducer.cpp.
struct ReducerBuffers {
    int32_t world;
    bool reduce_scatter;
    int32_t n_buckets;
    const int64_t *bucket_bytes;   // [n_buckets]
    const int64_t *bucket_flat;    // [n_buckets] byte offset in the flat buffers
    float *const *flat;            // [world], or NULL for a reducer without a device
    int device;
};
ReducerBuffers reducer_buffers(const ddp_reducer *r) noexcept;

}  // namespace ddp
