// paged_common.cuh -- index arithmetic and launches of the paged cache's kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

// A serving step is a chain of short kernels, and most of one's four microseconds
// are its launch.  The kernels of the paged cache are launched while the one
// before them in the stream still runs; each begins with chain_begin(), which
// waits until that one is done and its writes are visible, and lets the next one
// be launched: plan, append and decode of 64 tokens, one after the other, take
// 10.0 us instead of 16.4 launched by themselves and 8.0 instead of 9.3 in a graph.
// (A kernel that is not of this kind is waited for, and waits, as usual.)
// What a kernel reads may be written while it is on the GPU already: no load of such
// memory is a read-only one (__ldg).
__device__ __forceinline__ void chain_begin() {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int block, size_t smem,
                           cudaStream_t s, int cluster, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

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
