// tdp_rmsnorm.cu -- root-mean-square norm of rows with the residual's addition, in the plan's type or in 8 bits, its
// gradients, and the 8-bit form of rows that no norm makes.
//
// h = x + res, rounded as it is kept; rstd = 1 / sqrt(mean h^2 + eps), u = h * rstd, y = u * w.  With g = dy * w:
//   dx = dh + rstd * (g - u * mean(g * u)),  dw = sum over rows of dy * u.
// 8 bits (e4m3, a scale a row): v -> e4m3(448 v / m), m the row's largest |v|, scale m / 448.
//
// Bound by memory.  A row is read once: it stays in the registers of a team of lanes (a part of a warp, a warp, or up to
// eight warps) while its sums and its largest value are joined, 16-byte vectors lane after lane.  Teams walk over the rows
// with w in registers; the gradient keeps its sums for dw there too, joins a block's in shared memory and the blocks' in
// a second launch, in a fixed order.
#include <cuda_fp16.h>

#include <algorithm>

#include "tdp.h"
#include "tdp_internal.h"
#include "tdp_rows.cuh"

namespace {

constexpr int kNormThreads = 256;           // threads of a block at most: eight warps a row
constexpr int kNormVecs = 8;                // vectors of a lane at most
constexpr int kGradBlocks = 152 * 4;        // gradient: blocks at most, and so parts of dw
constexpr uint32_t kLeastBits = 0x0d800000u;        // 2^-100

struct norm_args {
    int64_t rows;
    int32_t C, nv;              // channels and 16-byte vectors of a row
    int32_t lanes;              // of a row: a power of two up to 32, or 32 times `warps`
    int32_t warps;              // of a row
    float eps, mean;            // mean: 1 / C
    const void *x, *res, *w;
    void *h, *y;
    float *rstd;
    uint8_t *y8, *x8;
    float *y8_scale, *x8_scale;
};

struct norm_grad_args {
    int64_t rows;
    int32_t C, nv, lanes, warps;
    float mean;
    const void *h, *w, *dy, *dh;
    const uint8_t *x8;
    const float *x8_scale, *rstd;
    void *dx;
    float *part;                // [blocks, C]
};

template <int N>
__device__ __forceinline__ void zero(float *f)
{
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = 0.f;
}

// Four values as e4m3, the first in the lowest byte; rounded to nearest even, past 448 to 448, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ void from_e4m3x4(uint32_t v, float *f)
{
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)v));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(v >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo)), b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

// A row's scale from the bits of its largest magnitude.  Magnitudes compare as integers, NaN above infinity above all else.
// A row that holds either has scale NaN, and NaN in every place; one below 2^-100 is counted as if that were its largest.
struct scale8 {
    float part, inv, scale;
    __device__ __forceinline__ explicit scale8(uint32_t top_bits)
    {
        const float top = top_bits >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __uint_as_float(max(top_bits, kLeastBits));
        part = top * (1.f / 512);
        inv = __frcp_rn(part);
        scale = __fdiv_rn(top, 448.f);
    }
    // 448 v / top as (0.875 v) / (top / 512): no product overflows and a value midway between two of e4m3's comes out
    // exact, so that it goes to the even one.  The quotient is corrected by its remainder (P. Markstein, "Computation of
    // elementary functions on the IBM RISC System/6000 processor", 1990): the plain product v * inv put 0.5 % of bf16's values
    // on the wrong side.
    __device__ __forceinline__ float of(float v) const
    {
        const float a = 0.875f * v, q = a * inv;
        return fmaf(fmaf(-q, part, a), inv, q);
    }
};

// V values of a row in 8 bits.
template <int V>
__device__ __forceinline__ void store8(uint8_t *p, const float *f, const scale8 &s)
{
    const uint32_t a = to_e4m3x4(s.of(f[0]), s.of(f[1]), s.of(f[2]), s.of(f[3]));
    if (V == 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(a, to_e4m3x4(s.of(f[V - 4]), s.of(f[V - 3]), s.of(f[V - 2]), s.of(f[V - 1])));
    } else {
        *reinterpret_cast<uint32_t *>(p) = a;
    }
}

// A thread's place: its row among those of a round, its lane in the row's team.
struct team {
    int32_t lane, row, rows;        // rows: of a block and round
    __device__ __forceinline__ explicit team(int32_t lanes)
    {
        row = threadIdx.x / lanes;
        lane = threadIdx.x - row * lanes;
        rows = blockDim.x / lanes;
    }
};

// Sum, and two maxima, over a row's team; every lane has the same.  `turn` changes from round to round.
__device__ __forceinline__ void join(int32_t lanes, int32_t warps, int32_t turn, float &sum, uint32_t &top, uint32_t &top2)
{
    __shared__ float ssum[2][kNormThreads / 32];
    __shared__ uint32_t stop[2][kNormThreads / 32], stop2[2][kNormThreads / 32];
    for (int32_t o = min(lanes, 32) / 2; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        top = max(top, __shfl_xor_sync(~0u, top, o));
        top2 = max(top2, __shfl_xor_sync(~0u, top2, o));
    }
    if (warps == 1) return;
    const int32_t k = turn & 1, w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
        ssum[k][w] = sum;
        stop[k][w] = top;
        stop2[k][w] = top2;
    }
    __syncthreads();            // the other half is written next: one barrier a round is enough
    sum = 0.f;
    top = top2 = 0;
    for (int32_t i = 0; i < warps; ++i) {
        sum += ssum[k][i];
        top = max(top, stop[k][i]);
        top2 = max(top2, stop2[k][i]);
    }
}

__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// NORM 0: the rows themselves, in 8 bits.  Q8: with outputs in 8 bits.
template <int BF16, int VPT, int NORM, int Q8>
__global__ void __launch_bounds__(kNormThreads)
tdp_rms_norm_kernel(const __grid_constant__ norm_args a)
{
    using E = tdp_elem<BF16>;
    constexpr int V = E::kVec;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const team t(a.lanes);
    const int64_t round = (int64_t)gridDim.x * t.rows;
    uint4 w[NORM ? VPT : 1];
    if (NORM && a.w) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            w[i] = c < a.nv ? static_cast<const uint4 *>(a.w)[c] : make_uint4(0, 0, 0, 0);
        }
    }
    // whole warps take part in every round, past the last row too
    const int64_t first = (int64_t)blockIdx.x * t.rows;
    int32_t turn = 0;
    for (int64_t r0 = first; r0 < a.rows; r0 += round, ++turn) {
        const int64_t r = r0 + t.row;
        const bool on = r < a.rows;
        const int64_t at = r * a.nv;
        uint4 x[VPT], s[NORM ? VPT : 1];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            const bool in = on && c < a.nv;
            x[i] = in ? __ldcs(static_cast<const uint4 *>(a.x) + at + c) : make_uint4(0, 0, 0, 0);
            if (NORM && a.res) s[i] = in ? __ldcs(static_cast<const uint4 *>(a.res) + at + c) : make_uint4(0, 0, 0, 0);
        }
        float sum = 0.f;
        uint32_t top = 0, top2 = 0;         // of |h w| and |h|
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            float f[V];
            E::unpack(x[i], f);
            if (NORM && a.res) {
                // rounded here, whether h is kept or not: the gradient reads it as it is kept, and is that of this function
                float g[V];
                E::unpack(s[i], g);
#pragma unroll
                for (int j = 0; j < V; ++j) f[j] += g[j];
                x[i] = E::pack(f);
                E::unpack(x[i], f);
            }
            if (NORM && a.h && on && c < a.nv) static_cast<uint4 *>(a.h)[at + c] = x[i];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (NORM) sum = fmaf(f[j], f[j], sum);
                if (Q8) top2 = max(top2, magnitude(f[j]));
            }
            if (NORM && Q8 && a.y8) {
                float g[V];
                if (a.w) E::unpack(w[i], g);
#pragma unroll
                for (int j = 0; j < V; ++j) top = max(top, magnitude(a.w ? f[j] * g[j] : f[j]));
            }
        }
        join(a.lanes, a.warps, turn, sum, top, top2);
        float rstd = 1.f;
        if (NORM) rstd = __frcp_rn(__fsqrt_rn(fmaf(sum, a.mean, a.eps)));
        if (NORM && a.rstd && on && t.lane == 0) a.rstd[r] = rstd;
        scale8 s8(0), u8(0);
        if (Q8 && NORM && a.y8) {
            s8 = scale8(magnitude(__uint_as_float(top) * rstd));
            if (on && t.lane == 0) a.y8_scale[r] = s8.scale;
        }
        if (Q8 && a.x8) {
            u8 = scale8(magnitude(__uint_as_float(top2) * rstd));
            if (on && t.lane == 0) a.x8_scale[r] = u8.scale;
        }
        if (!on) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            if (c >= a.nv) break;
            float f[V];
            E::unpack(x[i], f);
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] *= rstd;
            if (Q8 && a.x8) store8<V>(a.x8 + (at + c) * V, f, u8);
            if (NORM) {
                if (a.w) {
                    float g[V];
                    E::unpack(w[i], g);
#pragma unroll
                    for (int j = 0; j < V; ++j) f[j] *= g[j];
                }
                if (Q8 && a.y8) store8<V>(a.y8 + (at + c) * V, f, s8);
                if (a.y) static_cast<uint4 *>(a.y)[at + c] = E::pack(f);
            }
        }
    }
}

// KEPT8: u is x8 * x8_scale; otherwise h * rstd.
template <int BF16, int VPT, int KEPT8>
__global__ void __launch_bounds__(kNormThreads)
tdp_rms_norm_grad_kernel(const __grid_constant__ norm_grad_args a)
{
    using E = tdp_elem<BF16>;
    constexpr int V = E::kVec;
    extern __shared__ __align__(16) float acc[];        // [teams of a block, C]
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const team t(a.lanes);
    const int64_t round = (int64_t)gridDim.x * t.rows;
    uint4 w[VPT];
    float dw[VPT * V];
    zero<VPT * V>(dw);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int32_t c = t.lane + i * a.lanes;
        w[i] = a.w && c < a.nv ? static_cast<const uint4 *>(a.w)[c] : make_uint4(0, 0, 0, 0);
    }
    int32_t turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * t.rows; r0 < a.rows; r0 += round, ++turn) {
        const int64_t r = r0 + t.row;
        const bool on = r < a.rows;
        const int64_t at = r * a.nv;
        uint4 x[VPT], d[VPT], e[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            const bool in = on && c < a.nv;
            x[i] = d[i] = e[i] = make_uint4(0, 0, 0, 0);
            if (!in) continue;
            if (KEPT8) {
                if (V == 8) {
                    const uint2 p = __ldcs(reinterpret_cast<const uint2 *>(a.x8) + at + c);
                    x[i].x = p.x;
                    x[i].y = p.y;
                } else {
                    x[i].x = __ldcs(reinterpret_cast<const uint32_t *>(a.x8) + at + c);
                }
            } else {
                x[i] = __ldcs(static_cast<const uint4 *>(a.h) + at + c);
            }
            d[i] = __ldcs(static_cast<const uint4 *>(a.dy) + at + c);
            if (a.dh) e[i] = __ldcs(static_cast<const uint4 *>(a.dh) + at + c);
        }
        const float rstd = on ? a.rstd[r] : 0.f, unit = KEPT8 ? (on ? a.x8_scale[r] : 0.f) : rstd;
        auto rows = [&](int i, float *u, float *g) {
            if (KEPT8) {
                from_e4m3x4(x[i].x, u);
                if (V == 8) from_e4m3x4(x[i].y, u + V - 4);
            } else {
                E::unpack(x[i], u);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) u[j] *= unit;
            E::unpack(d[i], g);
        };
        float sum = 0.f;
        uint32_t no = 0, no2 = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float u[V], g[V], k[V];
            rows(i, u, g);
            if (a.w) E::unpack(w[i], k);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float p = g[j] * u[j];
                dw[i * V + j] += p;
                sum = a.w ? fmaf(p, k[j], sum) : sum + p;
            }
        }
        join(a.lanes, a.warps, turn, sum, no, no2);
        if (!on) continue;
        const float m = sum * a.mean;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            if (c >= a.nv) break;
            float u[V], g[V], k[V];
            rows(i, u, g);
            if (a.w) {
                E::unpack(w[i], k);
#pragma unroll
                for (int j = 0; j < V; ++j) g[j] *= k[j];
            }
            E::unpack(e[i], k);
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] = fmaf(fmaf(-u[j], m, g[j]), rstd, k[j]);
            static_cast<uint4 *>(a.dx)[at + c] = E::pack(g);
        }
    }
    if (!a.part) return;
    // a block's sums for dw, its teams' in order
    float *to = t.rows > 1 ? acc + t.row * a.C : a.part + (int64_t)blockIdx.x * a.C;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int32_t c = t.lane + i * a.lanes;
        if (c < a.nv) {
#pragma unroll
            for (int j = 0; j < V; j += 4) *reinterpret_cast<float4 *>(to + c * V + j) = make_float4(dw[i * V + j], dw[i * V + j + 1], dw[i * V + j + 2], dw[i * V + j + 3]);
        }
    }
    if (t.rows == 1) return;
    __syncthreads();
    for (int32_t c = threadIdx.x; c < a.C; c += blockDim.x) {
        float s = 0.f;
        for (int32_t k = 0; k < t.rows; ++k) s += acc[k * a.C + c];
        a.part[(int64_t)blockIdx.x * a.C + c] = s;
    }
}

// dw from the blocks' parts: 32 channels a block, the parts dealt to its warps.
__global__ void __launch_bounds__(1024)
tdp_rms_norm_dw_kernel(const float *part, int32_t parts, int32_t C, float *dw)
{
    __shared__ float s[32][33];
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float f = 0.f;
    if (c < C)
        for (int32_t p = warp; p < parts; p += 32) f += part[(int64_t)p * C + c];
    s[warp][lane] = f;
    __syncthreads();
    f = s[lane][warp];
    for (int o = 16; o; o >>= 1) f += __shfl_xor_sync(~0u, f, o);
    const int32_t mine = blockIdx.x * 32 + warp;
    if (lane == 0 && mine < C) dw[mine] = f;
}

// How rows are dealt to teams.
struct norm_shape {
    int32_t nv, vpt, lanes, warps, threads, rows;           // rows: of a block and round
};

norm_shape norm_deal(int32_t nv, int32_t most)
{
    norm_shape s;
    s.nv = nv;
    s.lanes = 1;
    while (s.lanes < 32 && s.lanes < nv) s.lanes *= 2;
    s.warps = std::max(1, (nv + 32 * most - 1) / (32 * most));
    s.lanes *= s.warps;
    const int32_t need = (nv + s.lanes - 1) / s.lanes;
    s.vpt = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : 8;
    s.threads = s.warps == 1 ? 128 : 32 * s.warps;
    s.rows = s.threads / s.lanes;
    return s;
}

tdp_status norm_check(tdp_plan_t plan, int64_t rows, int32_t C, int32_t *nv)
{
    if (!plan) return tdp_fail(TDP_ERR_INVALID_ARG, "null plan");
    if (rows < 0 || C < 1) return tdp_fail(TDP_ERR_INVALID_ARG, "need rows >= 0 and C >= 1");
    if (C > TDP_MAX_NORM_BYTES || (int64_t)C * plan->g.esize > TDP_MAX_NORM_BYTES)
        return tdp_fail(TDP_ERR_TOO_LARGE, "rows above TDP_MAX_NORM_BYTES");
    if (C * plan->g.esize % 16 != 0) return tdp_fail(TDP_ERR_MISALIGNED, "C * element size must be a multiple of 16 bytes");
    if (rows > ((int64_t)1 << 47)) return tdp_fail(TDP_ERR_TOO_LARGE, "rows above 2^47");
    *nv = C * plan->g.esize / 16;
    return TDP_OK;
}

template <int NORM, int Q8>
cudaError_t norm_launch(int bf16, const norm_shape &sh, const norm_args &a, cudaStream_t s)
{
    const unsigned grid = (unsigned)std::min<int64_t>((a.rows + sh.rows - 1) / sh.rows, 152 * (2048 / sh.threads));
#define TDP_NORM(V) \
    (bf16 ? tdp_launch(true, tdp_rms_norm_kernel<1, V, NORM, Q8>, grid, sh.threads, s, a) \
          : tdp_launch(true, tdp_rms_norm_kernel<0, V, NORM, Q8>, grid, sh.threads, s, a))
    return sh.vpt == 1 ? TDP_NORM(1) : sh.vpt == 2 ? TDP_NORM(2) : sh.vpt == 4 ? TDP_NORM(4) : TDP_NORM(8);
#undef TDP_NORM
}

// Blocks of the gradient; a block's sums for dw take `teams` rows of C floats in shared memory.
norm_shape grad_deal(int32_t nv, int32_t C, unsigned *grid, int64_t rows)
{
    norm_shape s = norm_deal(nv, kNormVecs);
    *grid = (unsigned)std::min<int64_t>((rows + s.rows - 1) / s.rows, kGradBlocks);
    return s;
}

}  // namespace

extern "C" tdp_status tdp_rms_norm(tdp_plan_t plan, int64_t rows, int32_t C, float eps, const void *x, const void *res,
                                   const void *w, void *h, void *y, float *rstd, uint8_t *y8, float *y8_scale, uint8_t *x8,
                                   float *x8_scale, tdp_stream_t stream)
{
    int32_t nv = 0;
    const tdp_status st = norm_check(plan, rows, C, &nv);
    if (st != TDP_OK) return st;
    if (!(eps >= 0.f) || eps - eps != 0.f) return tdp_fail(TDP_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (rows == 0) return tdp_ok();
    if (!x || (!y && !y8 && !x8 && !h && !rstd)) return tdp_fail(TDP_ERR_INVALID_ARG, "null x, or no output");
    if (!y8 != !y8_scale || !x8 != !x8_scale) return tdp_fail(TDP_ERR_INVALID_ARG, "8-bit rows and their scales come together");
    if (!tdp_aligned(x, 16) || !tdp_aligned(res, 16) || !tdp_aligned(w, 16) || !tdp_aligned(h, 16) || !tdp_aligned(y, 16) ||
        !tdp_aligned(y8, 16) || !tdp_aligned(x8, 16) || !tdp_aligned(rstd, 4) || !tdp_aligned(y8_scale, 4) || !tdp_aligned(x8_scale, 4))
        return tdp_fail(TDP_ERR_MISALIGNED, "rows and w need 16-byte, scales and rstd 4-byte alignment");
    const norm_shape sh = norm_deal(nv, kNormVecs);
    norm_args a = {rows, C, nv, sh.lanes, sh.warps, eps, 1.f / (float)C, x, res, w, h, y, rstd, y8, x8, y8_scale, x8_scale};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int bf16 = plan->g.dtype == TDP_BF16;
    const cudaError_t err = y8 || x8 ? norm_launch<1, 1>(bf16, sh, a, s) : norm_launch<1, 0>(bf16, sh, a, s);
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}

extern "C" tdp_status tdp_quant8(tdp_plan_t plan, int64_t rows, int32_t C, const void *x, uint8_t *x8, float *x8_scale,
                                 tdp_stream_t stream)
{
    int32_t nv = 0;
    const tdp_status st = norm_check(plan, rows, C, &nv);
    if (st != TDP_OK) return st;
    if (rows == 0) return tdp_ok();
    if (!x || !x8 || !x8_scale) return tdp_fail(TDP_ERR_INVALID_ARG, "null x, x8 or x8_scale");
    if (!tdp_aligned(x, 16) || !tdp_aligned(x8, 16) || !tdp_aligned(x8_scale, 4))
        return tdp_fail(TDP_ERR_MISALIGNED, "rows need 16-byte, scales 4-byte alignment");
    const norm_shape sh = norm_deal(nv, kNormVecs);
    norm_args a = {};
    a.rows = rows;
    a.C = C;
    a.nv = nv;
    a.lanes = sh.lanes;
    a.warps = sh.warps;
    a.x = x;
    a.x8 = x8;
    a.x8_scale = x8_scale;
    const cudaError_t err = norm_launch<0, 1>(plan->g.dtype == TDP_BF16, sh, a, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}

extern "C" tdp_status tdp_rms_norm_grad_workspace(tdp_plan_t plan, int64_t rows, int32_t C, int64_t *bytes)
{
    int32_t nv = 0;
    if (!bytes) return tdp_fail(TDP_ERR_INVALID_ARG, "null bytes");
    const tdp_status st = norm_check(plan, rows, C, &nv);
    if (st != TDP_OK) return st;
    unsigned grid = 0;
    grad_deal(nv, C, &grid, rows);
    *bytes = (int64_t)grid * C * 4;
    return tdp_ok();
}

extern "C" tdp_status tdp_rms_norm_grad(tdp_plan_t plan, int64_t rows, int32_t C, const void *h, const uint8_t *x8,
                                        const float *x8_scale, const float *rstd, const void *w, const void *dy,
                                        const void *dh, void *dx, float *dw, void *ws, int64_t ws_bytes, tdp_stream_t stream)
{
    int32_t nv = 0;
    const tdp_status st = norm_check(plan, rows, C, &nv);
    if (st != TDP_OK) return st;
    unsigned grid = 0;
    const norm_shape sh = grad_deal(nv, C, &grid, rows);
    if (rows > 0) {
        if (!rstd || !dy || !dx) return tdp_fail(TDP_ERR_INVALID_ARG, "null rstd, dy or dx");
        if (!h == !x8 || !x8 != !x8_scale) return tdp_fail(TDP_ERR_INVALID_ARG, "need h, or x8 with its scales, and not both");
        if (dw && (!ws || ws_bytes < (int64_t)grid * C * 4)) return tdp_fail(TDP_ERR_INVALID_ARG, "ws too small");
        if (!tdp_aligned(h, 16) || !tdp_aligned(x8, 16) || !tdp_aligned(w, 16) || !tdp_aligned(dy, 16) || !tdp_aligned(dh, 16) ||
            !tdp_aligned(dx, 16) || !tdp_aligned(x8_scale, 4) || !tdp_aligned(rstd, 4) || !tdp_aligned(ws, 256))
            return tdp_fail(TDP_ERR_MISALIGNED, "rows and w need 16-byte, scales and rstd 4-byte, ws 256-byte alignment");
    }
    if (!tdp_aligned(dw, 4)) return tdp_fail(TDP_ERR_MISALIGNED, "dw needs 4-byte alignment");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (rows > 0) {
        norm_grad_args a = {rows, C, nv, sh.lanes, sh.warps, 1.f / (float)C, h, w, dy, dh, x8, x8_scale, rstd, dx, dw ? static_cast<float *>(ws) : nullptr};
        const size_t smem = dw && sh.rows > 1 ? (size_t)sh.rows * C * 4 : 0;        // 32 KB at most
        const int bf16 = plan->g.dtype == TDP_BF16;
#define TDP_GRAD(V) \
    (bf16 ? (x8 ? tdp_launch_smem(true, tdp_rms_norm_grad_kernel<1, V, 1>, grid, sh.threads, smem, s, a) \
                : tdp_launch_smem(true, tdp_rms_norm_grad_kernel<1, V, 0>, grid, sh.threads, smem, s, a)) \
          : (x8 ? tdp_launch_smem(true, tdp_rms_norm_grad_kernel<0, V, 1>, grid, sh.threads, smem, s, a) \
                : tdp_launch_smem(true, tdp_rms_norm_grad_kernel<0, V, 0>, grid, sh.threads, smem, s, a)))
        err = sh.vpt == 1 ? TDP_GRAD(1) : sh.vpt == 2 ? TDP_GRAD(2) : sh.vpt == 4 ? TDP_GRAD(4) : TDP_GRAD(8);
#undef TDP_GRAD
    }
    if (err == cudaSuccess && dw)
        err = tdp_launch(true, tdp_rms_norm_dw_kernel, (unsigned)((C + 31) / 32), 1024, s, static_cast<const float *>(ws), (int32_t)grid, C, dw);
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}
