// Address ranges of the host sources' overlap checks. Not part of the C ABI.
#pragma once

#include <algorithm>
#include <cstdint>
#include <vector>

namespace ddp {

// Addresses [lo, hi).
struct Span {
    uintptr_t lo, hi;
};

// Sorted and apart.
using Spans = std::vector<Span>;

inline bool meets(const Spans &v, uintptr_t lo, uintptr_t hi)
{
    const auto it = std::partition_point(v.begin(), v.end(), [lo](const Span &s) { return s.hi <= lo; });
    return it != v.end() && it->lo < hi;
}

// Whether one of n rows of `bytes` bytes, `stride` bytes apart, the first at p,
// meets [lo, hi).
inline bool rows_meet(const void *p, int64_t n, int64_t stride, int64_t bytes, uintptr_t lo, uintptr_t hi)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    uintptr_t first = 0;   // the first row that ends past lo
    if (lo >= at + uintptr_t(bytes)) {
        if (stride == 0) return false;
        first = (lo - at - uintptr_t(bytes)) / uintptr_t(stride) + 1;
    }
    return first < uintptr_t(n) && at + first * uintptr_t(stride) < hi;
}

}  // namespace ddp
