// paged_common.cuh -- index arithmetic of the paged cache's kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

// n / P for 0 <= n < 2^31 as a product: with 2^(l-1) < P <= 2^l, M = ceil(2^(31+l) / P)
// overshoots by e < P <= 2^l parts in 2^(31+l), and n e < 2^(31+l).
struct Divide {
    uint32_t mul, shift, by;
};

inline Divide make_divide(uint32_t by) {
    uint32_t l = 0;
    while ((1ull << l) < by) ++l;
    const unsigned __int128 one = (unsigned __int128)1 << (31 + l);
    return {(uint32_t)((one + by - 1) / by), 31 + l, by};
}

__device__ __forceinline__ uint32_t divide(uint32_t n, const Divide &d) {
    return (uint32_t)(((uint64_t)n * d.mul) >> d.shift);
}

// a / b of non-negative numbers: in 32 bits, an eighth of the time, if they fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}
