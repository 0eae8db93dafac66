// tdp_host.h -- host-side helpers of the operators around the per-tile block (those of the tile path keep theirs in
// tdp_internal.h, whose bytes the recorded DRAM traffic of its kernels goes by).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

// Whether two buffers (either may be NULL) have a byte in common.
static inline bool tdp_overlap(const void *p, int64_t n, const void *q, int64_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}
// The same, but one buffer for both is fine.
static inline bool tdp_partly(const void *p, const void *q, int64_t n) { return p != q && tdp_overlap(p, n, q, n); }

// Raise a kernel's dynamic shared-memory limit once per device (`done`: one flag each).
template <typename K>
static inline cudaError_t tdp_allow_smem(K kernel, size_t bytes, std::atomic<bool> *done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_relaxed))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
    return e;
}
