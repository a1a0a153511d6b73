// Bounds on numbers that kernels read from device arrays.  Shared with the
// host, where the arithmetic can be checked.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define VLA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define VLA_HOST_DEVICE inline
#endif

namespace vla {

VLA_HOST_DEVICE int32_t bounded(int32_t x, int32_t low, int32_t high) {
    return x < low ? low : (x > high ? high : x);
}

// Rows begin .. end - 1 of a tensor of `total` rows, from two offsets of any
// value: 0 <= first, 0 <= n, first + n <= total.  The end is bounded before
// the difference is formed, which could pass 32 bits otherwise.
VLA_HOST_DEVICE void bounded_rows(int32_t begin, int32_t end, int32_t total, int32_t& first, int32_t& n) {
    first = bounded(begin, 0, total);
    n = bounded(end, first, total) - first;
}

}  // namespace vla
