// tdp_matmul8.cuh -- what the kernels of the product of 8-bit rows share.
#pragma once

#include "tdp_rows.cuh"
#include "tdp_tc.cuh"

namespace tdp_m8 {

using namespace tdp_tc;

constexpr int kK = 128;                     // values of K of a stage: a 128-byte row of a panel

struct args {
    const float *xs, *ws;       // scales of rows and of channels
    const void *bias, *res;
    void *out;
    int64_t rows;
    int32_t N, kb;              // channels, stages of K in all
    int32_t tiles_c;            // channel tiles
};

// Instruction descriptor: e4m3 x e4m3 -> fp32, M x N, both operands by rows.
constexpr uint32_t idesc8(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

// D[tmem] (+)= A B, K = 32; a and b are low words of descriptors.
__device__ __forceinline__ void mma8(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi)
        : "memory");
}

__device__ __forceinline__ void tma_load2(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Every thread of every block of the cluster.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// This block's shared address in block `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Waits, with a limit, for what is on its way to `bar`.
__device__ __forceinline__ void landed(uint32_t bar, uint32_t parity)
{
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitRounds && !mbar_try(bar, parity); ++i) {
    }
}

}  // namespace tdp_m8
