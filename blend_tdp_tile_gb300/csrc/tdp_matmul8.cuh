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
    int32_t tiles;              // pairs: tiles in all
    // Channels and rows of a load: fewer than a tile's where the product has fewer.  What a load fills with zeros past the end is slow
    // (12982 x 3328 x 32: 22.9 us where this takes 11.1); what it leaves out holds anything, and reaches only sums that nobody reads.
    int32_t w_box, x_box;
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

// Arrives at a barrier of any block of the cluster.
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// ------------------------------------------------------------------ pairs of blocks (cta_group::2)
__device__ __forceinline__ void pair_alloc(uint32_t slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_free(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// Box -> this block's shared memory, completing on a barrier of either block of the pair.
__device__ __forceinline__ void pair_load2(uint32_t dst, const CUtensorMap *map, uint32_t cluster_bar, int32_t x, int32_t y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
        : "memory");
}
// The product of the pair's tiles: each block holds half of A's rows, of B's and of D's, at the same addresses.
__device__ __forceinline__ void pair_mma8(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi)
        : "memory");
}
// One arrival at `bar` of both blocks when every product this thread has issued is done.
__device__ __forceinline__ void pair_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}
// Shared -> box of a tensor map.
__device__ __forceinline__ void tma_store2(const CUtensorMap *map, uint32_t src, int32_t x, int32_t y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the last store have been read.
__device__ __forceinline__ void tma_store_read_but_one() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

// Sums are 0 or from 2^-18 to 2^38 (products of e4m3, K of them at most): with a row's scale inside these bounds neither that product nor
// one with a channel's scale leaves fp32's range unless the result does.
__device__ __forceinline__ bool plain_scale(float xs) { return fabsf(xs) >= 0x1p-109f && fabsf(xs) <= 0x1p90f; }
// sum * xs * w + b for a row's scale outside them, by parts that stay inside.
__device__ __forceinline__ float far_scaled(float sum, float xs, float w, float b)
{
    const bool large = fabsf(xs) > 1.f, one = large ? fabsf(w) < 1.f : fabsf(w) > 1.f;        // one: the power of two that xs lacks goes to w
    const float up = large ? 0x1p64f : 0x1p-64f, down = large ? 0x1p-64f : 0x1p64f;
    return fmaf(sum * (xs * down) * (one ? w * up : w), one ? 1.f : up, b);
}

// Waits, with a limit, for what is on its way to `bar`.
__device__ __forceinline__ void landed(uint32_t bar, uint32_t parity)
{
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitRounds && !mbar_try(bar, parity); ++i) {
    }
}

}  // namespace tdp_m8
