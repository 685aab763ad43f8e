// page_math.cuh -- the sums that the page kernels share.
#pragma once

namespace svf {

__device__ __forceinline__ int sat_add(int a, int b, int cap) {
    // 0 <= a, b <= cap < 2^30: associative, so the order of a sum does not matter
    return min(a + b, cap);
}

__device__ __forceinline__ int pages_of(int tokens, int ps) {
    return tokens / ps + (tokens % ps != 0);
}

}  // namespace svf
