// api_checks.h -- what the argument checks of the C entry points share.
#pragma once
#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "gemm_nt.h"

namespace gnt {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Bytes [lo, hi) that an array of strided dimensions touches (at least one element each).
struct Span {
    uintptr_t lo, hi;
};
inline Span span_of(const void* base, int64_t esize, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1,
                    int64_t s2 = 0)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
    return {lo, lo + static_cast<uintptr_t>(((n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + 1) * esize)};
}
inline bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// Whether n0 x n1 x n2 elements with these strides end within 2^62 bytes (sizes are below 2^31).
inline bool in_range(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1, int64_t s2 = 0)
{
    const double e = static_cast<double>(n0) * static_cast<double>(s0) + static_cast<double>(n1) * static_cast<double>(s1) +
                     static_cast<double>(n2) * static_cast<double>(s2);
    return e * 4.0 < 4.0e18;
}

inline bool sizes_ok(std::initializer_list<int64_t> v)
{
    for (int64_t x : v)
        if (x < 0 || x > INT32_MAX)
            return false;
    return true;
}

inline gemm_status_t status_of(cudaError_t e) { return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

}  // namespace gnt
