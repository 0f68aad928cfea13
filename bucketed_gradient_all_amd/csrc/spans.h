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

}  // namespace ddp
