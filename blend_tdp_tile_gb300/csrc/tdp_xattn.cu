// tdp_xattn.cu -- cross attention of the tiles' tokens to an encoder's states, and its
// gradients: entry points and the fp32 kernels on the CUDA cores (bf16: tdp_xattn_tc.cuh, tdp_xattn_grad_tc.cuh).
//
// out = softmax(scale * Q K^T over the kept states) V, one pass over the states with the
// running maximum m and sum l of the softmax: a block holds 64 packed rows, takes 64
// states at a time, and rescales its sums by exp(m_old - m_new) when the maximum grows.  With
// few rows the states are split over blocks, whose outputs are joined by their log-sums.
// The gradient computes p = exp(s - lse) again: one kernel walks the states for dq,
// one walks the rows for dk and dv (split over the rows, joined in order: no
// atomics).  States that a row's mask drops are read as zero and get p = 0.
//
// The fp32 kernels are bound by instructions: each thread makes 4 x 4 scores from 8 loads of four elements.  35840 rows of
// 4 heads of 64 against 512 states take 649 us, 29 TFLOP/s, their gradients 2680 us, 25 TFLOP/s.
#include <algorithm>
#include <atomic>

#include "tdp.h"
#include "tdp_host.h"
#include "tdp_tensor_map.h"
#include "tdp_xattn.h"
#include "tdp_xattn_grad_tc.cuh"

namespace {

constexpr int kXT = 256;        // threads: 16 x 16, each 4 rows x 4 states
constexpr int kXM = 64;         // packed rows of a block
constexpr int kXN = 64;         // states of a step
constexpr int kXJoin = 64;      // threads of a join
constexpr float kLog2e = 1.4426950408889634f;

template <int DP>
struct xsm {
    static constexpr int kLd = DP + 4;      // row stride: lanes 4 banks apart
    static constexpr int kTile = 64 * kLd;
    static constexpr int kPs = kXN + 4;
};

// 64 rows of D elements to smem, zero past D and where row(i) gives NULL.
template <int DP, typename Row>
__device__ __forceinline__ void load_tile(float *dst, int32_t D, Row row)
{
    constexpr int NV = DP / 4;
    for (int32_t i = threadIdx.x; i < 64 * NV; i += kXT) {
        const int32_t r = i / NV, c = i % NV;
        const float *p = row(r);
        *reinterpret_cast<float4 *>(dst + r * xsm<DP>::kLd + c * 4) =
            p && c * 4 < D ? *reinterpret_cast<const float4 *>(p + c * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// acc[i][j] = A[4 ty + i] . B[tx + 16 j] over DP.
template <int DP>
__device__ __forceinline__ void dot_tile(const float *A, const float *B, int ty, int tx, float (&acc)[4][4])
{
    constexpr int L = xsm<DP>::kLd;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * L + d);
            y[i] = *reinterpret_cast<const float4 *>(B + (tx + 16 * i) * L + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
    }
}

// acc[i][4 c + e] += sum_j P[4 ty + i][j] * B[j][64 c + 4 tx + e]: rows of P times rows of B.
template <int DP>
__device__ __forceinline__ void mul_tile(const float *P, const float *B, int ty, int tx, float (&acc)[4][DP / 16])
{
    constexpr int L = xsm<DP>::kLd, LP = xsm<DP>::kPs;
#pragma unroll 2
    for (int j = 0; j < 64; j += 4) {
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(p[i]) = *reinterpret_cast<const float4 *>(P + (4 * ty + i) * LP + j);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int c = 0; c < DP / 64; ++c) {
                const float4 b = *reinterpret_cast<const float4 *>(B + (j + u) * L + 64 * c + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i][4 * c + 0] = fmaf(p[i][u], b.x, acc[i][4 * c + 0]);
                    acc[i][4 * c + 1] = fmaf(p[i][u], b.y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(p[i][u], b.z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(p[i][u], b.w, acc[i][4 * c + 3]);
                }
            }
    }
}

__device__ __forceinline__ float row_max16(float x)
{
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
    return x;
}
__device__ __forceinline__ float row_sum16(float x)
{
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

// Mask of the 64 states from s0 on: bit j of word j / 32.
__device__ __forceinline__ bool kept_bits(const uint8_t *mask, int32_t s0, int32_t S, uint32_t *bits)
{
    if (threadIdx.x < 64) {
        const int32_t s = s0 + threadIdx.x;
        const uint32_t w = __ballot_sync(~0u, s < S && (!mask || mask[s]));
        if ((threadIdx.x & 31) == 0) bits[threadIdx.x >> 5] = w;
    }
    __syncthreads();
    return (bits[0] | bits[1]) != 0;
}

// Offset of packed row r of key head kvh in rows and heads that lie `row` and `head` apart.
__device__ __forceinline__ int64_t packed(const xattn_args &a, const tdp_seg &seg, int32_t kvh, int64_t r, int64_t row,
                                          int64_t head)
{
    const int64_t tok = r / a.G;
    return (seg.row0 + tok) * row + (kvh * a.G + (int32_t)(r - tok * a.G)) * head;
}

// A row's log-sum; a row with no sum gets +inf, which makes its probabilities zero.
__device__ __forceinline__ float row_lse(float lse) { return lse == -INFINITY ? INFINITY : lse; }

template <int DP>
__global__ void __launch_bounds__(kXT)
tdp_xattn_simt_kernel(const __grid_constant__ tdp_geom g, const __grid_constant__ xattn_args a)
{
    extern __shared__ __align__(16) float sm[];
    float *Qs = sm, *Ks = Qs + xsm<DP>::kTile, *Vs = Ks + xsm<DP>::kTile, *Ps = Vs + xsm<DP>::kTile;
    __shared__ uint32_t bits[2];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int32_t w = blockIdx.x;
    const int32_t blk = w % a.blocks;
    w /= a.blocks;
    const int32_t kvh = w % a.Hkv;
    w /= a.Hkv;
    const int32_t part = w % a.split;
    const tdp_seg seg = xattn_seg(g, a, w / a.split);
    const int64_t r0 = (int64_t)blk * kXM, nr = seg.T * a.G - r0;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    if (nr <= 0) return;
    const uint8_t *mask = xattn_mask(a, g, seg);
    const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k) + seg.b * a.k_item + kvh * a.k_head,
            *v = static_cast<const float *>(a.v) + seg.b * a.v_item + kvh * a.v_head;
    load_tile<DP>(Qs, a.D, [&](int32_t r) { return r < nr ? q + packed(a, seg, kvh, r0 + r, a.q_row, a.q_head) : nullptr; });
    float m[4], l[4], acc[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
    }
    const float c2 = a.scale * kLog2e;
    const int32_t tile0 = part * a.part, tile1 = min((a.S + kXN - 1) / kXN, tile0 + a.part);
    for (int32_t t = tile0; t < tile1; ++t) {
        __syncthreads();
        if (!kept_bits(mask, t * kXN, a.S, bits)) continue;
        const uint32_t b0 = bits[0], b1 = bits[1];
        auto kept = [&](int32_t j) { return ((j < 32 ? b0 >> j : b1 >> (j - 32)) & 1) != 0; };
        load_tile<DP>(Ks, a.D, [&](int32_t j) { return kept(j) ? k + (int64_t)(t * kXN + j) * a.k_state : nullptr; });
        load_tile<DP>(Vs, a.D, [&](int32_t j) { return kept(j) ? v + (int64_t)(t * kXN + j) * a.v_state : nullptr; });
        __syncthreads();
        float s[4][4];
        dot_tile<DP>(Qs, Ks, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = kept(tx + 16 * j) ? s[i][j] * c2 : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
            const float mn = fmaxf(m[i], row_max16(top));
            const float base = mn == -INFINITY ? 0.f : mn, old = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                sum += p;
                Ps[(4 * ty + i) * xsm<DP>::kPs + tx + 16 * j] = p;
            }
            l[i] = l[i] * old + row_sum16(sum);
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) acc[i][c] *= old;
        }
        __syncwarp();       // a row's probabilities are written and read by one warp
        mul_tile<DP>(Ps, Vs, ty, tx, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t r = 4 * ty + i;
        if (r >= nr) continue;
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
        const float lse = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
        const int64_t h = packed(a, seg, kvh, r0 + r, a.Hq, 1);
        if (a.split > 1) {
            const int64_t at = (int64_t)part * a.rows * a.Hq + h;
            if (tx == 0) a.pl[at] = lse;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
                const int32_t d = 64 * (c / 4) + 4 * tx + c % 4;
                if (d < a.D) a.po[at * a.D + d] = acc[i][c] * inv;
            }
        } else {
            if (tx == 0 && a.lse) a.lse[h] = lse;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
                const int32_t d = 64 * (c / 4) + 4 * tx + c % 4;
                if (d < a.D) static_cast<float *>(a.out)[h * a.D + d] = acc[i][c] * inv;
            }
        }
    }
}

// One warp per (row, head), four columns a lane: out = sum_i exp(lse_i - lse) out_i over the parts of the states.
// A handful of warps in most cases, bound by latency: eight parts' loads run at a time, on as many SMs as there are.
template <int BF16>
__global__ void __launch_bounds__(kXJoin)
tdp_xattn_join_kernel(const xattn_args a)
{
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const int64_t n = a.rows * a.Hq, h = ((int64_t)blockIdx.x * kXJoin + threadIdx.x) >> 5;
    if (h >= n) return;
    const int32_t lane = threadIdx.x & 31;
    // a part's lse a lane (two past 32 parts)
    const float l0 = lane < a.split ? a.pl[lane * n + h] : -INFINITY, l1 = lane + 32 < a.split ? a.pl[(lane + 32) * n + h] : -INFINITY;
    float top = fmaxf(l0, l1);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float base = top == -INFINITY ? 0.f : top, w0 = expf(l0 - base), w1 = expf(l1 - base);
    float sum = w0 + w1;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const bool on = 4 * lane < a.D;
    const float *po = a.po + h * a.D + 4 * lane;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int32_t i = 0; i < a.split; ++i) {
        const float w = __shfl_sync(~0u, i < 32 ? w0 : w1, i & 31);
        const float4 x = on ? *reinterpret_cast<const float4 *>(po + i * n * a.D) : acc;
        if (w != 0.f) {
            acc.x += w * x.x;
            acc.y += w * x.y;
            acc.z += w * x.z;
            acc.w += w * x.w;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (on) {
        const int64_t at = h * a.D + 4 * lane;
        if (BF16)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
                make_uint2(tdp_pack_bf16x2(acc.x * inv, acc.y * inv), tdp_pack_bf16x2(acc.z * inv, acc.w * inv));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    if (lane == 0 && a.lse) a.lse[h] = sum == 0.f ? -INFINITY : base + logf(sum);
}

// dq of 64 packed rows, or a part of the states' share of it; delta = dout . out is written for the kernel that follows.
template <int DP>
__global__ void __launch_bounds__(kXT)
tdp_xattn_simt_dq_kernel(const __grid_constant__ tdp_geom g, const __grid_constant__ xattn_args a)
{
    extern __shared__ __align__(16) float sm[];
    float *Qs = sm, *Ds = Qs + xsm<DP>::kTile, *Ks = Ds + xsm<DP>::kTile, *Vs = Ks + xsm<DP>::kTile,
          *Ps = Vs + xsm<DP>::kTile;
    __shared__ uint32_t bits[2];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int32_t w = blockIdx.x;
    const int32_t blk = w % a.blocks;
    w /= a.blocks;
    const int32_t kvh = w % a.Hkv;
    w /= a.Hkv;
    const int32_t part = w % a.qsplit;
    const tdp_seg seg = xattn_seg(g, a, w / a.qsplit);
    const int64_t r0 = (int64_t)blk * kXM, nr = seg.T * a.G - r0;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    if (nr <= 0) return;
    const uint8_t *mask = xattn_mask(a, g, seg);
    const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k) + seg.b * a.k_item + kvh * a.k_head,
            *v = static_cast<const float *>(a.v) + seg.b * a.v_item + kvh * a.v_head;
    auto row = [&](const void *p, int32_t r) -> const float * {
        return r < nr ? static_cast<const float *>(p) + packed(a, seg, kvh, r0 + r, (int64_t)a.Hq * a.D, a.D) : nullptr;
    };
    load_tile<DP>(Qs, a.D, [&](int32_t r) { return row(a.o, r); });
    load_tile<DP>(Ds, a.D, [&](int32_t r) { return row(a.dout, r); });
    __syncthreads();
    float lse[4], delta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float d = 0.f;
        for (int c = tx; c < DP; c += 16) d += Qs[(4 * ty + i) * xsm<DP>::kLd + c] * Ds[(4 * ty + i) * xsm<DP>::kLd + c];
        delta[i] = row_sum16(d);
        const int32_t r = 4 * ty + i;
        lse[i] = INFINITY;
        if (r < nr) {
            const int64_t h = packed(a, seg, kvh, r0 + r, a.Hq, 1);
            lse[i] = row_lse(a.lse[h]);
            if (tx == 0 && part == 0) a.delta[h] = delta[i];
        }
    }
    __syncthreads();
    load_tile<DP>(Qs, a.D, [&](int32_t r) { return r < nr ? q + packed(a, seg, kvh, r0 + r, a.q_row, a.q_head) : nullptr; });
    float acc[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
    const int32_t last = min((a.S + kXN - 1) / kXN, (part + 1) * a.qpart);
    for (int32_t t = part * a.qpart; t < last; ++t) {
        __syncthreads();
        if (!kept_bits(mask, t * kXN, a.S, bits)) continue;
        const uint32_t b0 = bits[0], b1 = bits[1];
        auto kept = [&](int32_t j) { return ((j < 32 ? b0 >> j : b1 >> (j - 32)) & 1) != 0; };
        load_tile<DP>(Ks, a.D, [&](int32_t j) { return kept(j) ? k + (int64_t)(t * kXN + j) * a.k_state : nullptr; });
        load_tile<DP>(Vs, a.D, [&](int32_t j) { return kept(j) ? v + (int64_t)(t * kXN + j) * a.v_state : nullptr; });
        __syncthreads();
        float s[4][4], dp[4][4];
        dot_tile<DP>(Qs, Ks, ty, tx, s);
        dot_tile<DP>(Ds, Vs, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                Ps[(4 * ty + i) * xsm<DP>::kPs + tx + 16 * j] =
                    kept(tx + 16 * j) ? expf(fmaf(s[i][j], a.scale, -lse[i])) * (dp[i][j] - delta[i]) * a.scale : 0.f;
        __syncwarp();
        mul_tile<DP>(Ps, Ks, ty, tx, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t r = 4 * ty + i;
        if (r >= nr) continue;
        float *o = const_cast<float *>(a.qsplit > 1 ? row(a.pq + part * a.rows * a.Hq * a.D, r) : row(a.dq, r));
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const int32_t d = 64 * (c / 4) + 4 * tx + c % 4;
            if (d < a.D) o[d] = acc[i][c];
        }
    }
}

// dk and dv of 64 states: the transposed tiles, states as rows, over a part of the row blocks of
// every segment of the item.
template <int DP>
__global__ void __launch_bounds__(kXT)
tdp_xattn_simt_dkv_kernel(const __grid_constant__ tdp_geom g, const __grid_constant__ xattn_args a)
{
    extern __shared__ __align__(16) float sm[];
    float *Ks = sm, *Vs = Ks + xsm<DP>::kTile, *Qs = Vs + xsm<DP>::kTile, *Ds = Qs + xsm<DP>::kTile,
          *Ps = Ds + xsm<DP>::kTile, *Ss = Ps + 64 * xsm<DP>::kPs;
    __shared__ uint32_t bits[2];
    __shared__ float row_ls[kXM], row_delta[kXM];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t tiles = (a.S + kXN - 1) / kXN;
    int32_t w = blockIdx.x;
    const int32_t t = w % tiles;
    w /= tiles;
    const int32_t kvh = w % a.Hkv;
    w /= a.Hkv;
    const int32_t part = w % a.split, b = w / a.split;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k) + b * a.k_item + kvh * a.k_head,
            *v = static_cast<const float *>(a.v) + b * a.v_item + kvh * a.v_head;
    // a state no mask of its segments keeps is never multiplied by a kept probability, but
    // another tile's may keep it: the tiles are loaded as they are and selected per segment
    load_tile<DP>(Ks, a.D, [&](int32_t j) { return t * kXN + j < a.S ? k + (int64_t)(t * kXN + j) * a.k_state : nullptr; });
    load_tile<DP>(Vs, a.D, [&](int32_t j) { return t * kXN + j < a.S ? v + (int64_t)(t * kXN + j) * a.v_state : nullptr; });
    float dk[4][DP / 16], dv[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
    const int32_t nsegs = a.flat ? 1 : g.nt;
    const int64_t first = (int64_t)part * a.part, last = min((int64_t)nsegs * a.blocks, first + a.part);
    int32_t cur = -1;
    bool any = false;
    tdp_seg seg = {};
    for (int64_t u = first; u < last; ++u) {
        const int32_t sg = (int32_t)(u / a.blocks);
        const int64_t r0 = (u % a.blocks) * kXM;
        if (sg != cur) {
            cur = sg;
            seg = xattn_seg(g, a, sg * g.B + b);
            __syncthreads();
            any = kept_bits(xattn_mask(a, g, seg), t * kXN, a.S, bits);
        }
        const int64_t nr = seg.T * a.G - r0;
        if (!any || nr <= 0) continue;
        const uint32_t b0 = bits[0], b1 = bits[1];
        auto kept = [&](int32_t j) { return ((j < 32 ? b0 >> j : b1 >> (j - 32)) & 1) != 0; };
        __syncthreads();
        load_tile<DP>(Qs, a.D, [&](int32_t r) { return r < nr ? q + packed(a, seg, kvh, r0 + r, a.q_row, a.q_head) : nullptr; });
        load_tile<DP>(Ds, a.D, [&](int32_t r) {
            return r < nr ? static_cast<const float *>(a.dout) + packed(a, seg, kvh, r0 + r, (int64_t)a.Hq * a.D, a.D) : nullptr;
        });
        if (threadIdx.x < kXM) {
            float ls = INFINITY, de = 0.f;
            if (threadIdx.x < nr) {
                const int64_t h = packed(a, seg, kvh, r0 + threadIdx.x, a.Hq, 1);
                ls = row_lse(a.lse[h]);
                de = a.delta[h];
            }
            row_ls[threadIdx.x] = ls;
            row_delta[threadIdx.x] = de;
        }
        __syncthreads();
        float s[4][4], dp[4][4];
        dot_tile<DP>(Ks, Qs, ty, tx, s);
        dot_tile<DP>(Vs, Ds, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t r = tx + 16 * j;
                const bool on = kept(4 * ty + i);
                const float p = on ? expf(fmaf(s[i][j], a.scale, -row_ls[r])) : 0.f;
                Ps[(4 * ty + i) * xsm<DP>::kPs + r] = p;
                Ss[(4 * ty + i) * xsm<DP>::kPs + r] = on ? p * (dp[i][j] - row_delta[r]) * a.scale : 0.f;
            }
        __syncwarp();
        mul_tile<DP>(Ps, Ds, ty, tx, dv);
        mul_tile<DP>(Ss, Qs, ty, tx, dk);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t st = t * kXN + 4 * ty + i;
        if (st >= a.S) continue;
        const int64_t at = (((int64_t)b * a.S + st) * a.Hkv + kvh) * a.D, all = (int64_t)part * g.B * a.S * a.Hkv * a.D;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const int32_t d = 64 * (c / 4) + 4 * tx + c % 4;
            if (d >= a.D) continue;
            if (a.split > 1) {
                a.pk[all + at + d] = dk[i][c];
                a.pv[all + at + d] = dv[i][c];
            } else {
                static_cast<float *>(a.dk)[at + d] = dk[i][c];
                static_cast<float *>(a.dv)[at + d] = dv[i][c];
            }
        }
    }
}

// fp32 dq from its parts, four elements a thread, parts in order.
__global__ void __launch_bounds__(kXT)
tdp_xattn_dq_join_kernel(const xattn_args a, int64_t n)
{
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const int64_t i = ((int64_t)blockIdx.x * kXT + threadIdx.x) * 4;
    if (i >= n) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int32_t k = 0; k < a.qsplit; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(a.pq + k * n + i);
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    }
    *reinterpret_cast<float4 *>(static_cast<float *>(a.dq) + i) = s;
}

// dk and dv from their parts, four elements a thread, parts in order.
template <int BF16>
__global__ void __launch_bounds__(kXT)
tdp_xattn_dkv_join_kernel(const xattn_args a, int64_t n)
{
    using T = typename tdp_elem<BF16>::type;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const int64_t i = ((int64_t)blockIdx.x * kXT + threadIdx.x) * 4;
    if (i >= 2 * n) return;
    const float *p = i < n ? a.pk + i : a.pv + (i - n);
    T *o = i < n ? static_cast<T *>(a.dk) + i : static_cast<T *>(a.dv) + (i - n);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int32_t k = 0; k < a.split; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(p + k * n);
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    }
    o[0] = (T)s.x;
    o[1] = (T)s.y;
    o[2] = (T)s.z;
    o[3] = (T)s.w;
}

constexpr int kSplitMax = 64;  // two parts a lane in the join
// fp32: blocks below which the work is split, two for each SM.  Eight items of one token, 5000 states: 76 us against 680
// unsplit; dk and dv of 512 states from 35840 rows: 2683 us against 12016; gradients of 64 rows, 4 heads of 128,
// 3000 states, 174 us against 747 with dq unsplit.
constexpr int kFill = 304;
constexpr int kSMs = 152;       // what splits are chosen for
// Items of a launch, parts included (what is split has few): blocks that step through them pass the end by less than the rest.
constexpr int64_t kMostItems = 0x7fffffffLL - 65536;

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// The launches' shapes and the workspace's layout.
struct xattn_shape {
    int64_t mask_rows, kept_bytes;          // bf16: lists of kept state tiles
    int64_t fwd_bytes, grad_bytes;
    int64_t pl_at, po_at;                   // forward
    int64_t delta_at, pk_at, pv_at, pq_at;  // gradient
    int32_t fblocks, fsplit, fpart;
    int32_t bblocks, bsplit, bpart;
};

// Parts of `tiles` state tiles for `items` row blocks, fewer than the device's SMs: as many as make the device's
// rounds of blocks, each as long as its tiles and one more, take the least time.  (Few rows are bound by
// reading the states, which goes on from one block's item to the next.)  Eight items of one token, 32 heads on 8, 8192
// states: 68 us against 76 in one part (64 blocks).
int32_t split_states(int64_t items, int64_t tiles)
{
    if (items == 0 || items >= kSMs || tiles < 2) return 1;
    int64_t best = 0;
    int32_t split = 1;
    for (int32_t s = 1; s <= std::min<int64_t>(kSplitMax, tiles); ++s) {
        const int64_t cost = (items * s + kSMs - 1) / kSMs * ((tiles + s - 1) / s + 1) + (s > 1 ? 3 : 0);
        if (s == 1 || cost <= best) {
            best = cost;
            split = s;
        }
    }
    return split;
}

// Parts of the row blocks of a state tile (dk, dv; bf16): the device's rounds of blocks, each as long as its
// row tiles and about three more, against the parts' way through memory (16 bytes an element written and read,
// in row-tile times of 1.1 us).  35840 rows of 16 heads of 128 on 4, 640 states: gradients in 476 us against 1779 in one
// part (20 blocks); 16 heads of 64, 1000 states (128 blocks): 515 against 509.
int64_t split_rows(int64_t base, int64_t units, int64_t heads, int64_t elements)
{
    int64_t split = 1;
    double best = 0.;
    for (int64_t s = 1; s <= std::min<int64_t>(kSplitMax, units); ++s) {
        const double cost = (double)((base * s + kSMs - 1) / kSMs) * (double)((units + s - 1) / s * heads + 3) +
                            (s > 1 ? (double)s * (double)elements * 2.1e-6 + 3. : 0.);
        if (s == 1 || cost < best) {
            best = cost;
            split = s;
        }
    }
    return split;
}

tdp_status xattn_check(tdp_plan_t plan, const tdp_xattn *p, xattn_args *a, xattn_shape *sh)
{
    if (!plan || !p) return tdp_fail(TDP_ERR_INVALID_ARG, "null plan or shape");
    const tdp_geom &g = plan->g;
    if (p->q_heads < 1 || p->kv_heads < 1 || p->q_heads % p->kv_heads != 0 || p->head_dim < 1 || p->states < 0)
        return tdp_fail(TDP_ERR_INVALID_ARG, "need heads >= 1, q_heads a multiple of kv_heads, head_dim >= 1 and states >= 0");
    if (!(p->scale == p->scale) || p->scale - p->scale != 0.f)
        return tdp_fail(TDP_ERR_INVALID_ARG, "scale must be finite");
    if (p->head_dim > TDP_MAX_HEAD_DIM || p->states > TDP_MAX_STATES)
        return tdp_fail(TDP_ERR_TOO_LARGE, "head_dim above TDP_MAX_HEAD_DIM or states above TDP_MAX_STATES");
    const int64_t strides[8] = {p->q_row, p->q_head, p->k_item, p->k_state, p->k_head, p->v_item, p->v_state, p->v_head};
    const int64_t V = 16 / g.esize;
    if (p->head_dim % V != 0) return tdp_fail(TDP_ERR_MISALIGNED, "head_dim * element size must be a multiple of 16 bytes");
    for (int64_t s : strides) {
        if (s < 0) return tdp_fail(TDP_ERR_INVALID_ARG, "strides must not be negative");
        if (s % V != 0) return tdp_fail(TDP_ERR_MISALIGNED, "strides must be multiples of 16 bytes");
        if (s >= ((int64_t)1 << 38)) return tdp_fail(TDP_ERR_TOO_LARGE, "strides must be below 2^38 elements");
    }
    if ((p->q_row == 0 && (int64_t)g.B * g.total > 1) || (p->q_head == 0 && p->q_heads > 1) ||
        ((p->k_state == 0 || p->v_state == 0) && p->states > 1))
        return tdp_fail(TDP_ERR_INVALID_ARG, "rows, query heads and states cannot be broadcast (stride 0)");
    *a = xattn_args{};
    a->q_row = p->q_row;
    a->q_head = p->q_head;
    a->k_item = p->k_item;
    a->k_state = p->k_state;
    a->k_head = p->k_head;
    a->v_item = p->v_item;
    a->v_state = p->v_state;
    a->v_head = p->v_head;
    a->rows = (int64_t)g.B * g.total;
    a->Hq = p->q_heads;
    a->Hkv = p->kv_heads;
    a->G = p->q_heads / p->kv_heads;
    a->D = p->head_dim;
    a->S = p->states;
    a->scale = p->scale;
    a->per_tile = p->mask_per_tile != 0 && g.nt > 1;
    a->flat = g.B == 1 && !a->per_tile;
    a->segs = a->flat ? 1 : g.nt * g.B;
    const int64_t T = a->flat ? a->rows : tdp_max_tile_tokens(g);
    if (a->rows > 0x7fffffffLL / a->Hq) return tdp_fail(TDP_ERR_TOO_LARGE, "rows * q_heads must be below 2^31");
    a->blocks = (int32_t)((T * a->G + kXM - 1) / kXM);
    const bool bf16 = g.dtype == TDP_BF16;
    const int64_t tiles = (a->S + kXN - 1) / kXN, tiles128 = (a->S + tdp_xt::kKeys - 1) / tdp_xt::kKeys;
    const int64_t grid = (int64_t)a->segs * a->Hkv * a->blocks, kvgrid = (int64_t)g.B * a->Hkv * tiles;
    sh->mask_rows = a->per_tile ? (int64_t)g.nt * g.B : g.B;
    sh->kept_bytes = bf16 ? 2 * align256(sh->mask_rows * tiles128 * 16) + align256(sh->mask_rows * tiles128 * 4) + 2 * align256(sh->mask_rows * 4) : 0;
    sh->fsplit = 1;
    sh->fpart = (int32_t)std::max<int64_t>(tiles, 1);
    if (bf16) {
        a->Gp = std::min(a->G, 128);
        while (a->G % a->Gp != 0) --a->Gp;
        a->TT = 128 / a->Gp;
        sh->fblocks = (int32_t)((T + 2 * a->TT - 1) / (2 * a->TT));
        const int64_t items = (int64_t)a->segs * (a->Hq / a->Gp) * sh->fblocks;
        if (items > kMostItems) return tdp_fail(TDP_ERR_TOO_LARGE, "cross attention grid too large");
        sh->fsplit = split_states(items, tiles128);
        a->by_heads = fast_div_by(a->Hq / a->Gp);
        a->by_group = fast_div_by(a->G);
        a->by_B = fast_div_by(std::max(g.B, 1));
        a->by_nH = fast_div_by(g.d[1].n);
        a->by_nW = fast_div_by(g.d[2].n);
    } else {
        if (grid > kMostItems || kvgrid > kMostItems) return tdp_fail(TDP_ERR_TOO_LARGE, "cross attention grid too large");
        // few row blocks: the states in parts of four tiles or more, few enough to fill the device
        sh->fblocks = a->blocks;
        if (grid > 0 && grid < kFill && tiles > 4) {
            const int64_t want = std::min<int64_t>({kSplitMax, (kFill + grid - 1) / grid, tiles / 4});
            sh->fpart = (int32_t)((tiles + want - 1) / want);
            sh->fsplit = (int32_t)((tiles + sh->fpart - 1) / sh->fpart);
        }
    }
    // few state tiles: the row blocks in parts
    sh->bblocks = bf16 ? (int32_t)((T + a->TT - 1) / a->TT) : a->blocks;
    const int64_t units = (int64_t)(a->flat ? 1 : g.nt) * sh->bblocks;
    sh->bsplit = 1;
    sh->bpart = (int32_t)std::max<int64_t>(units, 1);
    if (bf16) {
        const int64_t base = (int64_t)g.B * a->Hkv * tiles128, hbs = a->G / a->Gp;
        if (units > kMostItems || base > kMostItems || (int64_t)a->segs * (a->Hq / a->Gp) * sh->bblocks > kMostItems)
            return tdp_fail(TDP_ERR_TOO_LARGE, "cross attention grid too large");
        const int64_t s = split_rows(base, units, hbs, (int64_t)g.B * a->S * a->Hkv * a->D);
        sh->bpart = (int32_t)std::max<int64_t>((units + s - 1) / s, 1);
        sh->bsplit = (int32_t)std::max<int64_t>((units + sh->bpart - 1) / sh->bpart, 1);
        if (base * sh->bsplit > kMostItems) return tdp_fail(TDP_ERR_TOO_LARGE, "cross attention grid too large");
    } else if (kvgrid > 0 && kvgrid < kFill && units > 1) {
        const int64_t want = std::min<int64_t>({kSplitMax, (kFill + kvgrid - 1) / kvgrid, units});
        sh->bpart = (int32_t)((units + want - 1) / want);
        sh->bsplit = (int32_t)((units + sh->bpart - 1) / sh->bpart);
    }
    const int64_t rh = a->rows * a->Hq, kv = (int64_t)g.B * a->S * a->Hkv * a->D;
    sh->pl_at = sh->kept_bytes;
    sh->po_at = sh->pl_at + (sh->fsplit > 1 ? align256(sh->fsplit * rh * 4) : 0);
    sh->fwd_bytes = sh->po_at + (sh->fsplit > 1 ? sh->fsplit * rh * a->D * 4 : 0);
    sh->delta_at = sh->kept_bytes;
    sh->pk_at = sh->delta_at + align256(rh * 4);
    sh->pv_at = sh->pk_at + (sh->bsplit > 1 ? align256(sh->bsplit * kv * 4) : 0);
    sh->pq_at = sh->pv_at + (sh->bsplit > 1 ? align256(sh->bsplit * kv * 4) : 0);
    // fp32: dq splits the states as the forward does
    a->qsplit = bf16 ? 1 : sh->fsplit;
    a->qpart = sh->fpart;
    sh->grad_bytes = sh->pq_at + (a->qsplit > 1 ? a->qsplit * rh * a->D * 4 : 0);
    return TDP_OK;
}

// Multiprocessors of the current device, asked once.
int sm_count()
{
    static std::atomic<int> count[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return kSMs;
    if (dev < 64 && (n = count[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return kSMs;
    if (dev < 64) count[dev].store(n, std::memory_order_relaxed);
    return n;
}

// bf16: the lists of kept tiles, then the product kernel.
cudaError_t tc_kept(const xattn_shape &sh, xattn_args *a, unsigned char *ws, cudaStream_t s)
{
    const int64_t tiles = (a->S + tdp_xt::kKeys - 1) / tdp_xt::kKeys;
    a->kept_words = reinterpret_cast<uint4 *>(ws);
    a->kept_tile = reinterpret_cast<int32_t *>(ws + align256(sh.mask_rows * tiles * 16));
    a->kept_n = reinterpret_cast<int32_t *>(ws + align256(sh.mask_rows * tiles * 16) + align256(sh.mask_rows * tiles * 4));
    a->kept_states = a->kept_n + align256(sh.mask_rows * 4) / 4;
    a->state_words = reinterpret_cast<uint4 *>(ws + sh.kept_bytes - align256(sh.mask_rows * tiles * 16));
    if (!a->mask) return cudaSuccess;
    const unsigned threads = (unsigned)std::min<int64_t>(1024, 32 * std::max<int64_t>(tiles, 1));
    return tdp_launch(true, tdp_xt::tdp_xattn_kept_kernel, (unsigned)sh.mask_rows, threads, s, a->mask, a->S, a->kept_n, a->kept_states, a->kept_tile, a->kept_words, a->state_words);
}

// Tensor map of bf16 rows: `dims` extents from the contiguous one on, strides and box of them.  A dimension of
// one, or one that is broadcast (stride 0), has the smallest stride a map takes and is read at coordinate 0.
bool tc_map(CUtensorMap *map, const void *p, int dims, const int64_t *extent, const int64_t *stride, const int64_t *box)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = tdp_encode_tiled();
    if (!encode) return false;
    cuuint64_t e[5], st[4];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < dims; ++i) {
        e[i] = i > 0 && stride[i] == 0 ? 1 : (cuuint64_t)std::max<int64_t>(extent[i], 1);
        b[i] = (cuuint32_t)box[i];
        one[i] = 1;
        if (i > 0) st[i - 1] = (cuuint64_t)(stride[i] > 0 ? stride[i] * 2 : 16);
    }
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void *>(p), e, st, b, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Maps of q-like rows [R, Hq, D] (a tile: Gp heads of TT tokens) and of states [B, S, Hkv, D] (128 states of a head).
bool tc_row_map(CUtensorMap *map, const void *p, const xattn_args &a, int64_t row, int64_t head)
{
    const int64_t extent[3] = {a.D, a.Hq, a.rows}, stride[3] = {1, head, row}, box[3] = {64, a.Gp, a.TT};
    return tc_map(map, p, 3, extent, stride, box);
}
bool tc_state_map(CUtensorMap *map, const void *p, const tdp_geom &g, const xattn_args &a, int64_t item, int64_t state, int64_t head)
{
    const int64_t extent[4] = {a.D, a.Hkv, a.S, g.B}, stride[4] = {1, head, state, item}, box[4] = {64, 1, tdp_xt::kKeys, 1};
    return tc_map(map, p, 4, extent, stride, box);
}

template <int DP>
cudaError_t tc_forward(const tdp_geom &g, const xattn_args &a, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    constexpr size_t bytes = tdp_xt::fwd_smem<DP>::kBytes;
    cudaError_t e = tdp_allow_smem(tdp_xt::tdp_xattn_tc_kernel<DP>, bytes, done);
    CUtensorMap q, k, v, o;
    // with no states the kernel loads nothing: q stands in for the maps of k and v
    if (e == cudaSuccess &&
        (!tc_row_map(&q, a.q, a, a.q_row, a.q_head) || !tc_row_map(&o, a.out, a, (int64_t)a.Hq * a.D, a.D) ||
         !tc_state_map(&k, a.S > 0 ? a.k : a.q, g, a, a.k_item, a.k_state, a.k_head) ||
         !tc_state_map(&v, a.S > 0 ? a.v : a.q, g, a, a.v_item, a.v_state, a.v_head)))
        e = cudaErrorInvalidValue;
    const int32_t items = a.segs * a.split * (a.Hq / a.Gp) * a.blocks;
    if (e == cudaSuccess)
        e = tdp_launch_smem(true, tdp_xt::tdp_xattn_tc_kernel<DP>, (unsigned)std::min(items, sm_count()), tdp_xt::kThreads, bytes, s, g, a, q, k, v, o, items);
    return e;
}

template <int DP>
cudaError_t tc_grad(const tdp_geom &g, const xattn_args &a, cudaStream_t s)
{
    static std::atomic<bool> done_q[64], done_kv[64];
    constexpr size_t bytes_q = tdp_xt::dq_smem<DP>::kBytes, bytes_kv = tdp_xt::dkv_smem<DP>::kBytes;
    cudaError_t e = tdp_allow_smem(tdp_xt::tdp_xattn_dq_kernel<DP>, bytes_q, done_q);
    if (e == cudaSuccess) e = tdp_allow_smem(tdp_xt::tdp_xattn_dkv_kernel<DP>, bytes_kv, done_kv);
    CUtensorMap q, o, d, k, v;
    const int64_t row = (int64_t)a.Hq * a.D;
    if (e == cudaSuccess &&
        (!tc_row_map(&q, a.q, a, a.q_row, a.q_head) || !tc_row_map(&o, a.o, a, row, a.D) || !tc_row_map(&d, a.dout, a, row, a.D) ||
         !tc_state_map(&k, a.S > 0 ? a.k : a.q, g, a, a.k_item, a.k_state, a.k_head) ||
         !tc_state_map(&v, a.S > 0 ? a.v : a.q, g, a, a.v_item, a.v_state, a.v_head)))
        e = cudaErrorInvalidValue;
    const int32_t items = a.segs * (a.Hq / a.Gp) * a.blocks;
    if (e == cudaSuccess)
        e = tdp_launch_smem(true, tdp_xt::tdp_xattn_dq_kernel<DP>, (unsigned)std::min(items, sm_count()), tdp_xt::kThreads, bytes_q, s, g, a, q, o, d, k, v, items);
    const unsigned grid = (unsigned)(g.B * a.split * a.Hkv * ((a.S + tdp_xt::kKeys - 1) / tdp_xt::kKeys));
    if (e == cudaSuccess && a.S > 0)
        e = tdp_launch_smem(true, tdp_xt::tdp_xattn_dkv_kernel<DP>, grid, tdp_xt::kThreads, bytes_kv, s, g, a, q, d, k, v);
    return e;
}

template <int DP>
struct simt_kernels {
    static constexpr size_t kFwd = (3 * xsm<DP>::kTile + 64 * xsm<DP>::kPs) * 4;
    static constexpr size_t kDq = (4 * xsm<DP>::kTile + 64 * xsm<DP>::kPs) * 4;
    static constexpr size_t kDkv = (4 * xsm<DP>::kTile + 2 * 64 * xsm<DP>::kPs) * 4;
    // Raise the kernels' dynamic shared-memory limits once per device.
    static cudaError_t prepare()
    {
        static std::atomic<bool> done[64];
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_relaxed))) return e;
        const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
        e = cudaFuncSetAttribute(tdp_xattn_simt_kernel<DP>, attr, (int)kFwd);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(tdp_xattn_simt_dq_kernel<DP>, attr, (int)kDq);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(tdp_xattn_simt_dkv_kernel<DP>, attr, (int)kDkv);
        if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
        return e;
    }
    static cudaError_t forward(const tdp_geom &g, const xattn_args &a, cudaStream_t s)
    {
        cudaError_t e = prepare();
        if (e == cudaSuccess)
            e = tdp_launch_smem(true, tdp_xattn_simt_kernel<DP>, (unsigned)(a.segs * a.split * a.Hkv * a.blocks), kXT, kFwd, s, g, a);
        return e;
    }
    static cudaError_t dq(const tdp_geom &g, const xattn_args &a, cudaStream_t s)
    {
        cudaError_t e = prepare();
        if (e == cudaSuccess)
            e = tdp_launch_smem(true, tdp_xattn_simt_dq_kernel<DP>, (unsigned)(a.segs * a.qsplit * a.Hkv * a.blocks), kXT, kDq, s, g, a);
        return e;
    }
    static cudaError_t dkv(const tdp_geom &g, const xattn_args &a, cudaStream_t s)
    {
        const unsigned grid = (unsigned)(g.B * a.split * a.Hkv * ((a.S + kXN - 1) / kXN));
        return tdp_launch_smem(true, tdp_xattn_simt_dkv_kernel<DP>, grid, kXT, kDkv, s, g, a);
    }
};

}  // namespace

extern "C" tdp_status tdp_cross_attn_workspace(tdp_plan_t plan, const tdp_xattn *p, int32_t grad, int64_t *bytes)
{
    xattn_args a;
    xattn_shape sh;
    if (!bytes) return tdp_fail(TDP_ERR_INVALID_ARG, "null bytes");
    const tdp_status st = xattn_check(plan, p, &a, &sh);
    if (st != TDP_OK) return st;
    *bytes = grad ? sh.grad_bytes : sh.fwd_bytes;
    return tdp_ok();
}

extern "C" tdp_status tdp_cross_attn(tdp_plan_t plan, const tdp_xattn *p, const void *q, const void *k, const void *v,
                                     const uint8_t *mask, void *out, float *lse, void *ws, int64_t ws_bytes,
                                     tdp_stream_t stream)
{
    xattn_args a;
    xattn_shape sh;
    const tdp_status st = xattn_check(plan, p, &a, &sh);
    if (st != TDP_OK) return st;
    const tdp_geom &g = plan->g;
    if (g.B == 0) return tdp_ok();
    if (!q || !out || (a.S > 0 && (!k || !v)) || (sh.fwd_bytes > 0 && (!ws || ws_bytes < sh.fwd_bytes)))
        return tdp_fail(TDP_ERR_INVALID_ARG, "null q, k, v or out, or ws too small");
    if (!tdp_aligned(q, 16) || !tdp_aligned(k, 16) || !tdp_aligned(v, 16) || !tdp_aligned(out, 16) ||
        !tdp_aligned(lse, 4) || !tdp_aligned(ws, 256))
        return tdp_fail(TDP_ERR_MISALIGNED, "q, k, v and out need 16-byte, lse 4-byte, ws 256-byte alignment");
    a.q = q;
    a.k = k;
    a.v = v;
    a.mask = mask;
    a.out = out;
    a.lse = lse;
    a.split = sh.fsplit;
    a.part = sh.fpart;
    a.blocks = sh.fblocks;
    a.by_blocks = fast_div_by(a.blocks);
    a.by_split = fast_div_by(a.split);
    unsigned char *w = reinterpret_cast<unsigned char *>(ws);
    a.pl = reinterpret_cast<float *>(w + sh.pl_at);
    a.po = reinterpret_cast<float *>(w + sh.po_at);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (g.dtype == TDP_BF16) {
        err = tc_kept(sh, &a, w, s);
        // heads to 64 columns have kernels of their own: 156 us, gradients 515, against 200 and 693 in those for 128
        // (35840 rows, 16 heads of 64, 1000 states)
        if (err == cudaSuccess) err = a.D <= 64 ? tc_forward<64>(g, a, s) : tc_forward<128>(g, a, s);
    } else {
        err = a.D <= 64 ? simt_kernels<64>::forward(g, a, s) : simt_kernels<128>::forward(g, a, s);
    }
    if (err == cudaSuccess && a.split > 1) {
        const unsigned grid = (unsigned)((a.rows * a.Hq * 32 + kXJoin - 1) / kXJoin);
        err = g.dtype == TDP_BF16 ? tdp_launch(true, tdp_xattn_join_kernel<1>, grid, kXJoin, s, a)
                                  : tdp_launch(true, tdp_xattn_join_kernel<0>, grid, kXJoin, s, a);
    }
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}

extern "C" tdp_status tdp_cross_attn_grad(tdp_plan_t plan, const tdp_xattn *p, const void *q, const void *k,
                                          const void *v, const uint8_t *mask, const void *out, const float *lse,
                                          const void *dout, void *dq, void *dk, void *dv, void *ws, int64_t ws_bytes,
                                          tdp_stream_t stream)
{
    xattn_args a;
    xattn_shape sh;
    const tdp_status st = xattn_check(plan, p, &a, &sh);
    if (st != TDP_OK) return st;
    const tdp_geom &g = plan->g;
    if (g.B == 0) return tdp_ok();
    if (!q || !out || !lse || !dout || !dq || (a.S > 0 && (!k || !v || !dk || !dv)) || !ws || ws_bytes < sh.grad_bytes)
        return tdp_fail(TDP_ERR_INVALID_ARG, "null buffer, or ws too small");
    if (!tdp_aligned(q, 16) || !tdp_aligned(k, 16) || !tdp_aligned(v, 16) || !tdp_aligned(out, 16) ||
        !tdp_aligned(dout, 16) || !tdp_aligned(dq, 16) || !tdp_aligned(dk, 16) || !tdp_aligned(dv, 16) ||
        !tdp_aligned(lse, 4) || !tdp_aligned(ws, 256))
        return tdp_fail(TDP_ERR_MISALIGNED, "elements need 16-byte, lse 4-byte, ws 256-byte alignment");
    a.q = q;
    a.k = k;
    a.v = v;
    a.mask = mask;
    a.o = out;
    a.lse = const_cast<float *>(lse);
    a.dout = dout;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    unsigned char *w = reinterpret_cast<unsigned char *>(ws);
    a.delta = reinterpret_cast<float *>(w + sh.delta_at);
    a.pk = reinterpret_cast<float *>(w + sh.pk_at);
    a.pv = reinterpret_cast<float *>(w + sh.pv_at);
    a.pq = reinterpret_cast<float *>(w + sh.pq_at);
    a.split = sh.bsplit;
    a.part = sh.bpart;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (g.dtype == TDP_BF16) {
        a.blocks = sh.bblocks;
        a.by_blocks = fast_div_by(a.blocks);
        err = tc_kept(sh, &a, w, s);
        if (err == cudaSuccess) err = a.D <= 64 ? tc_grad<64>(g, a, s) : tc_grad<128>(g, a, s);
    } else {
        err = a.D <= 64 ? simt_kernels<64>::dq(g, a, s) : simt_kernels<128>::dq(g, a, s);
        if (err == cudaSuccess && a.S > 0) err = a.D <= 64 ? simt_kernels<64>::dkv(g, a, s) : simt_kernels<128>::dkv(g, a, s);
    }
    if (err == cudaSuccess && a.S > 0) {
        if (err == cudaSuccess && a.split > 1) {
            const int64_t n = (int64_t)g.B * a.S * a.Hkv * a.D;
            const unsigned grid = (unsigned)((2 * n / 4 + kXT - 1) / kXT);
            err = g.dtype == TDP_BF16 ? tdp_launch(true, tdp_xattn_dkv_join_kernel<1>, grid, kXT, s, a, n)
                                      : tdp_launch(true, tdp_xattn_dkv_join_kernel<0>, grid, kXT, s, a, n);
        }
        if (err == cudaSuccess && a.qsplit > 1) {
            const int64_t n = a.rows * a.Hq * a.D;
            err = tdp_launch(true, tdp_xattn_dq_join_kernel, (unsigned)((n / 4 + kXT - 1) / kXT), kXT, s, a, n);
        }
    }
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}
