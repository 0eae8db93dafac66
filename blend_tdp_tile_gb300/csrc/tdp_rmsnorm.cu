// tdp_rmsnorm.cu -- root-mean-square norm of rows with the residual's addition, in the plan's type or in 8 bits, its
// gradients, and the 8-bit form of rows that no norm makes.
//
// h = x + res, rounded as it is kept; rstd = 1 / sqrt(mean h^2 + eps), u = h * rstd, y = u * w.  With g = dy * w:
//   dx = dh + rstd * (g - u * mean(g * u)),  dw = sum over rows of dy * u.
// 8 bits (e4m3, a scale a row): v -> e4m3(448 v / m), m the row's largest |v|, scale m / 448.
//
// Bound by memory.  A row is read once: a team of lanes (a part of a warp, a warp, or up to eight warps) brings it to shared
// memory, each lane its own 16-byte vectors, a row ahead, some 100 KB an SM on their way; sums and largest
// values are joined over the team, and the second pass reads shared memory or registers.  Nobody but the lane itself reads its
// vectors, so no barrier stands between a copy and its use.  The gradient keeps its sums for dw in registers over all its rows, joins
// a block's in shared memory and the blocks' in a second launch, in a fixed order.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "tdp.h"
#include "tdp_host.h"
#include "tdp_internal.h"
#include "tdp_rows.cuh"
#include "tdp_tc.cuh"

namespace {

using tdp_tc::add2;
using tdp_tc::fma2;
using tdp_tc::mul2;
using tdp_tc::pair;
using tdp_tc::unpair;

// Threads of a block at most: a lane's registers hold its vectors, and in the gradient their sums for dw.
constexpr int kNormThreads = 512;
constexpr int norm_threads(int vpt, bool grad) { return vpt <= (grad ? 4 : 6) ? kNormThreads : 256; }
constexpr int kNormWarps = 8;               // warps of a row at most
constexpr int kNormVecs = 6, kGradVecs = 4; // vectors of a lane, forward and gradient (eight where eight warps need them)
constexpr int kSMs = 152;
constexpr int kNormSmem = 196608;           // bytes of rows that an SM has on their way and at work
constexpr float kLeast = 0x1p-100f;

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

// B bytes to shared memory on their way, zeros where `on` is false.
template <int B>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool on)
{
    const int n = on ? B : 0;
    if (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(B) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Largest magnitude; NaN goes before all else.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A vector of the plan's type as pairs of fp32, and back.
template <int BF16>
__device__ __forceinline__ void pairs_of(const uint4 &u, uint64_t *p)
{
    float f[8];
    tdp_elem<BF16>::unpack(u, f);
#pragma unroll
    for (int j = 0; j < tdp_elem<BF16>::kVec / 2; ++j) p[j] = pair(f[2 * j], f[2 * j + 1]);
}
template <int BF16>
__device__ __forceinline__ uint4 of_pairs(const uint64_t *p)
{
    float f[8];
#pragma unroll
    for (int j = 0; j < tdp_elem<BF16>::kVec / 2; ++j) unpair(p[j], f[2 * j], f[2 * j + 1]);
    return tdp_elem<BF16>::pack(f);
}
template <int P>
__device__ __forceinline__ void top_of(const uint64_t *p, float &top)
{
#pragma unroll
    for (int j = 0; j < P; ++j) {
        float a, b;
        unpair(p[j], a, b);
        top = max_nan(top, max_nan(fabsf(a), fabsf(b)));
    }
}

// Two pairs as e4m3, the first in the lowest byte; rounded to nearest even, past 448 to 448, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(uint64_t p, uint64_t q)
{
    float a, b, c, d;
    unpair(p, a, b);
    unpair(q, c, d);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ void from_e4m3x4(uint32_t v, uint64_t *p)
{
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)v));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(v >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo)), b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
    p[0] = pair(a.x, a.y);
    p[1] = pair(b.x, b.y);
}
template <int P>
__device__ __forceinline__ void store8(uint8_t *p, const uint64_t *v)
{
    const uint32_t a = to_e4m3x4(v[0], v[1]);
    if (P == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(a, to_e4m3x4(v[P - 2], v[P - 1]));
    else *reinterpret_cast<uint32_t *>(p) = a;
}

// The largest magnitude that a row's scale is made of: NaN for a row that holds NaN or an infinity, which then has scale NaN
// and NaN in every place; 2^-100 for less.
__device__ __forceinline__ float top8(float top) { return top < INFINITY ? fmaxf(top, kLeast) : NAN; }

// How a norm's rows v rstd become e4m3: 448 v rstd / m.  m is rstd times the row's largest |v|, `top`, so rstd cancels and 448 v / top
// is left, a quotient of numbers as they came: of bf16 rows (h, or h w, which fp32 holds) often midway between two of e4m3's.  The
// factor is kept in two parts, so that one rounding is left and such a value stays where it is and goes to the even one; a product
// with the first part alone puts 0.05 % of x8's values on the wrong side.
struct code8 {
    uint64_t k, rest;
    // y = top * rstd, m = top8(y); lift: what v is multiplied by before, 1 or 2^100.  top * lift is 2^-118 at least, or y below 2^-100.
    __device__ __forceinline__ void make(float top, float rstd, float y, float m, float lift)
    {
        const float den = m < INFINITY ? top * lift : NAN;
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(den * (1 / 64.f)));      // neither is too small for fp32
        float f = inv * 7.f, r = fmaf(-f, den, 448.f) * (inv * (1 / 64.f));
        if (y < kLeast) {           // m counts as 2^-100
            f = 448.f / kLeast / lift * rstd;
            r = 0.f;
        }
        k = pair(f, f);
        rest = pair(r, r);
    }
    template <int P>
    __device__ __forceinline__ void of(uint64_t *v) const
    {
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = fma2(v[j], k, mul2(v[j], rest));
    }
};

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
template <int TOP>
__device__ __forceinline__ void join(int32_t lanes, int32_t warps, int32_t turn, float &sum, float &top, float &top2)
{
    __shared__ float ssum[2][kNormThreads / 32], stop[2][TOP ? kNormThreads / 32 : 1], stop2[2][TOP ? kNormThreads / 32 : 1];
    for (int32_t o = min(lanes, 32) / 2; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        if (TOP) {
            top = max_nan(top, __shfl_xor_sync(~0u, top, o));
            top2 = max_nan(top2, __shfl_xor_sync(~0u, top2, o));
        }
    }
    if (warps == 1) return;
    const int32_t k = turn & 1, w = threadIdx.x >> 5, first = w - w % warps;
    if ((threadIdx.x & 31) == 0) {
        ssum[k][w] = sum;
        if (TOP) {
            stop[k][w] = top;
            stop2[k][w] = top2;
        }
    }
    // the team's own barrier; the other half is written next: one a round is enough
    asm volatile("bar.sync %0, %1;" ::"r"(1 + first), "r"(lanes) : "memory");
    sum = 0.f;
    top = top2 = 0.f;
    for (int32_t i = 0; i < warps; ++i) {
        sum += ssum[k][first + i];
        if (TOP) {
            top = max_nan(top, stop[k][first + i]);
            top2 = max_nan(top2, stop2[k][first + i]);
        }
    }
}

// What is written in 8 bits: nothing; the checkpoint x8 and no y8; y8, or both; the same where eps leaves rstd above 2^18 (see
// code8::make).  The checkpoint has a form of its own as y goes with it: 168960 rows of 2048 bf16 take 272 us by it and 338 by the next.
enum { kPlain = 0, kKept8 = 1, kAny8 = 2, kSmall8 = 3 };

// NORM 0: the rows themselves, in 8 bits.  RES: with a residual.
template <int BF16, int VPT, int NORM, int Q8, int RES>
__global__ void __launch_bounds__(norm_threads(VPT, false))
tdp_rms_norm_kernel(const __grid_constant__ norm_args a)
{
    using E = tdp_elem<BF16>;
    constexpr int V = E::kVec, P = V / 2, IN = 1 + RES, S = 2;       // inputs, rows in shared memory
    constexpr bool Y8 = Q8 >= kAny8, SMALL = Q8 == kSmall8;
    extern __shared__ __align__(16) uint4 slots[];      // [S][IN][VPT][threads]
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const team t(a.lanes);
    const int64_t round = (int64_t)gridDim.x * t.rows;
    const int32_t threads = blockDim.x;
    const uint4 *mine = slots + threadIdx.x;
    auto bring = [&](int64_t r0, int32_t stage) {
        const int64_t r = r0 + t.row;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            const bool on = r < a.rows && c < a.nv;
            const int64_t at = on ? r * a.nv + c : 0;
            const uint32_t to = tdp_tc::smem_u32(mine + (stage * IN * VPT + i) * threads);
            copy_async<16>(to, static_cast<const uint4 *>(a.x) + at, on);
            if (RES) copy_async<16>(to + VPT * threads * 16, static_cast<const uint4 *>(a.res) + at, on);
        }
        copy_commit();
    };
    const int64_t first = (int64_t)blockIdx.x * t.rows;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) bring(first + s * round, s);
    uint4 w[NORM ? VPT : 1];
    if (NORM && a.w) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            w[i] = c < a.nv ? static_cast<const uint4 *>(a.w)[c] : make_uint4(0, 0, 0, 0);
        }
    }
    // whole warps take part in every round, past the last row too
    int32_t turn = 0, stage = 0;
    for (int64_t r0 = first; r0 < a.rows; r0 += round, ++turn) {
        bring(r0 + (S - 1) * round, stage == 0 ? S - 1 : stage - 1);
        copy_wait<S - 1>();
        const int64_t r = r0 + t.row;
        const bool on = r < a.rows;
        const int64_t at = r * a.nv;
        uint4 x[VPT];
        uint64_t sum2 = 0;
        float top = 0.f, top2 = 0.f;            // of |h w| and |h|
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            uint64_t f[P];
            x[i] = mine[(stage * IN * VPT + i) * threads];
            pairs_of<BF16>(x[i], f);
            if (RES) {
                // rounded here, whether h is kept or not: the gradient reads it as it is kept, and is that of this function
                uint64_t g[P];
                pairs_of<BF16>(mine[((stage * IN + 1) * VPT + i) * threads], g);
#pragma unroll
                for (int j = 0; j < P; ++j) f[j] = add2(f[j], g[j]);
                x[i] = of_pairs<BF16>(f);
                if (BF16) pairs_of<BF16>(x[i], f);
            }
            if (NORM && a.h && on && c < a.nv) static_cast<uint4 *>(a.h)[at + c] = x[i];
            if (NORM) {
#pragma unroll
                for (int j = 0; j < P; ++j) sum2 = fma2(f[j], f[j], sum2);
            }
            if (Q8 && (!NORM || !Y8 || a.x8)) top_of<P>(f, top2);
            if (NORM && Y8 && a.y8) {
                if (a.w) {
                    uint64_t g[P];
                    pairs_of<BF16>(w[i], g);
#pragma unroll
                    for (int j = 0; j < P; ++j) f[j] = mul2(f[j], g[j]);
                }
                top_of<P>(f, top);
            }
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        float sum, other;
        unpair(sum2, sum, other);
        sum += other;
        join<Q8>(a.lanes, a.warps, turn, sum, top, top2);
        const float rstd = NORM ? __frcp_rn(__fsqrt_rn(fmaf(sum, a.mean, a.eps))) : 1.f;
        if (NORM && a.rstd && on && t.lane == 0) a.rstd[r] = rstd;
        float part = 0.f, inv = 0.f;
        code8 cy = {}, cx = {};
        const float lift_y = SMALL && top < kLeast ? 1 / kLeast : 1.f, lift_x = SMALL && top2 < kLeast ? 1 / kLeast : 1.f;
        if (Y8 && NORM && a.y8) {
            const float y = top * rstd, m = top8(y);
            if (on && t.lane == 0) a.y8_scale[r] = __fdiv_rn(m, 448.f);
            cy.make(top, rstd, y, m, lift_y);
        }
        if (Q8 && (!Y8 || a.x8)) {
            if (NORM) {
                const float y = top2 * rstd, m = top8(y);
                if (on && t.lane == 0) a.x8_scale[r] = __fdiv_rn(m, 448.f);
                cx.make(top2, rstd, y, m, lift_x);
            } else {
                const float m = top8(top2);
                if (on && t.lane == 0) a.x8_scale[r] = __fdiv_rn(m, 448.f);
                part = -m * (1.f / 512);
                inv = __frcp_rn(-part);
            }
        }
        if (!on) continue;
        const uint64_t rs = pair(rstd, rstd);
        // y beside y8: h rstd before w, as without 8 bits.  Within the loop below it costs calls without y a tenth; before it, more
        // than four vectors a lane want more registers than there are, and behind it 168960 x 2048 with a residual take 2 % longer.
        auto plain = [&] {
            if (!NORM || !Y8 || !a.y) return;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int32_t c = t.lane + i * a.lanes;
                if (c >= a.nv) break;
                uint64_t f[P], g[P];
                pairs_of<BF16>(x[i], f);
                if (a.w) pairs_of<BF16>(w[i], g);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    f[j] = mul2(f[j], rs);
                    if (a.w) f[j] = mul2(f[j], g[j]);
                }
                static_cast<uint4 *>(a.y)[at + c] = of_pairs<BF16>(f);
            }
        };
        if (VPT <= 4) plain();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            if (c >= a.nv) break;
            uint64_t f[P], q[P];
            // h w is made again: carried over from the first pass in registers, 8192 channels take 25 % longer
            if (Y8 && VPT > 4) asm volatile("" : "+r"(x[i].x), "+r"(x[i].y), "+r"(x[i].z), "+r"(x[i].w));
            pairs_of<BF16>(x[i], f);
            if (!NORM) {
                // 448 v / m as (0.875 v) / (m / 512): no product overflows and a value midway between two of e4m3's comes out
                // exact, so that it goes to the even one.  The quotient is corrected by its remainder (P. Markstein, "Computation of
                // elementary functions on the IBM RISC System/6000 processor", 1990): the plain product v * inv put 0.5 % of
                // bf16's values on the wrong side.
                const uint64_t e = pair(0.875f, 0.875f), n = pair(part, part), k = pair(inv, inv);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const uint64_t v = mul2(f[j], e);
                    q[j] = mul2(v, k);
                    q[j] = fma2(fma2(q[j], n, v), k, q[j]);
                }
                store8<P>(a.x8 + (at + c) * V, q);
                continue;
            }
            if (Q8 && (!Y8 || a.x8)) {
#pragma unroll
                for (int j = 0; j < P; ++j) q[j] = SMALL ? mul2(f[j], pair(lift_x, lift_x)) : f[j];
                cx.of<P>(q);
                store8<P>(a.x8 + (at + c) * V, q);
            }
            if (!Y8) {
#pragma unroll
                for (int j = 0; j < P; ++j) f[j] = mul2(f[j], rs);
            }
            if (a.w) {
                uint64_t g[P];
                pairs_of<BF16>(w[i], g);
#pragma unroll
                for (int j = 0; j < P; ++j) f[j] = mul2(f[j], g[j]);
            }
            if (Y8 && a.y8) {
#pragma unroll
                for (int j = 0; j < P; ++j) q[j] = SMALL ? mul2(f[j], pair(lift_y, lift_y)) : f[j];
                cy.of<P>(q);
                store8<P>(a.y8 + (at + c) * V, q);
            }
            if (!Y8 && a.y) static_cast<uint4 *>(a.y)[at + c] = of_pairs<BF16>(f);
        }
        if (VPT > 4) plain();
    }
    copy_wait<0>();
}

// KEPT8: u is x8 * x8_scale; otherwise h * rstd.  The rows stay in shared memory for the second pass.
template <int BF16, int VPT, int KEPT8>
__global__ void __launch_bounds__(norm_threads(VPT, true))
tdp_rms_norm_grad_kernel(const __grid_constant__ norm_grad_args a)
{
    using E = tdp_elem<BF16>;
    constexpr int V = E::kVec, P = V / 2, IN = 3, S = 2;
    extern __shared__ __align__(16) uint4 slots[];      // [S][IN][VPT][threads]; at the end [teams of a block, C] sums
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const team t(a.lanes);
    const int64_t round = (int64_t)gridDim.x * t.rows;
    const int32_t threads = blockDim.x;
    const uint4 *mine = slots + threadIdx.x;
    auto bring = [&](int64_t r0, int32_t stage) {
        const int64_t r = r0 + t.row;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int32_t c = t.lane + i * a.lanes;
            const bool on = r < a.rows && c < a.nv;
            const int64_t at = on ? r * a.nv + c : 0;
            const uint32_t to = tdp_tc::smem_u32(mine + (stage * IN * VPT + i) * threads);
            if (KEPT8) copy_async<V>(to, a.x8 + at * V, on);
            else copy_async<16>(to, static_cast<const uint4 *>(a.h) + at, on);
            copy_async<16>(to + VPT * threads * 16, static_cast<const uint4 *>(a.dy) + at, on);
            if (a.dh) copy_async<16>(to + 2 * VPT * threads * 16, static_cast<const uint4 *>(a.dh) + at, on);
        }
        copy_commit();
    };
    const int64_t first = (int64_t)blockIdx.x * t.rows;
    bring(first, 0);
    uint4 w[VPT];
    uint64_t dw[VPT * P];
#pragma unroll
    for (int i = 0; i < VPT * P; ++i) dw[i] = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int32_t c = t.lane + i * a.lanes;
        w[i] = a.w && c < a.nv ? static_cast<const uint4 *>(a.w)[c] : make_uint4(0, 0, 0, 0);
    }
    int32_t turn = 0;
    for (int64_t r0 = first; r0 < a.rows; r0 += round, ++turn) {
        const int32_t stage = turn & 1;
        const int64_t r = r0 + t.row;
        const bool on = r < a.rows;
        const float rstd = on ? a.rstd[r] : 0.f, unit = KEPT8 ? (on ? a.x8_scale[r] : 0.f) : rstd;
        bring(r0 + round, stage ^ 1);
        copy_wait<1>();
        auto row = [&](int i, uint64_t *u, uint64_t *g) {
            const uint4 *at = mine + (stage * IN * VPT + i) * threads;
            if (KEPT8) {
                const uint2 p = *reinterpret_cast<const uint2 *>(at);
                from_e4m3x4(p.x, u);
                if (V == 8) from_e4m3x4(p.y, u + P - 2);
            } else {
                pairs_of<BF16>(*at, u);
            }
            pairs_of<BF16>(at[VPT * threads], g);
        };
        uint64_t sum2 = 0;
        const uint64_t un = pair(unit, unit);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            uint64_t u[P], g[P], k[P];
            row(i, u, g);
            if (a.w) pairs_of<BF16>(w[i], k);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const uint64_t p = mul2(g[j], mul2(u[j], un));
                dw[i * P + j] = add2(dw[i * P + j], p);
                sum2 = a.w ? fma2(p, k[j], sum2) : add2(sum2, p);
            }
        }
        float sum, other, no = 0.f, no2 = 0.f;
        unpair(sum2, sum, other);
        sum += other;
        join<0>(a.lanes, a.warps, turn, sum, no, no2);
        if (on) {
            const float m = -sum * a.mean * unit;
            const uint64_t m2 = pair(m, m), rs = pair(rstd, rstd);
            uint4 *dx = static_cast<uint4 *>(a.dx) + r * a.nv;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int32_t c = t.lane + i * a.lanes;
                if (c >= a.nv) break;
                uint64_t u[P], g[P], k[P];
                row(i, u, g);
                if (a.w) {
                    pairs_of<BF16>(w[i], k);
#pragma unroll
                    for (int j = 0; j < P; ++j) g[j] = mul2(g[j], k[j]);
                }
                if (a.dh) {
                    pairs_of<BF16>(mine[((stage * IN + 2) * VPT + i) * threads], k);
                } else {
#pragma unroll
                    for (int j = 0; j < P; ++j) k[j] = 0;
                }
#pragma unroll
                for (int j = 0; j < P; ++j) g[j] = fma2(fma2(u[j], m2, g[j]), rs, k[j]);
                dx[c] = of_pairs<BF16>(g);
            }
        }
    }
    copy_wait<0>();
    if (!a.part) return;
    // a block's sums for dw, its teams' in order
    if (t.rows > 1) __syncthreads();
    float *acc = reinterpret_cast<float *>(slots);
    float *to = t.rows > 1 ? acc + t.row * a.C : a.part + (int64_t)blockIdx.x * a.C;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int32_t c = t.lane + i * a.lanes;
        if (c < a.nv) {
#pragma unroll
            for (int j = 0; j < P; j += 2) *reinterpret_cast<ulonglong2 *>(to + c * V + 2 * j) = make_ulonglong2(dw[i * P + j], dw[i * P + j + 1]);
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
    constexpr int U = 16;               // parts whose loads a thread has under way: a warp's share is 10 to 38
    for (int32_t p0 = warp; p0 < parts; p0 += 32 * U) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = c < C && p0 + 32 * u < parts ? part[(int64_t)(p0 + 32 * u) * C + c] : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) f += v[u];
    }
    s[warp][lane] = f;
    __syncthreads();
    f = s[lane][warp];
    for (int o = 16; o; o >>= 1) f += __shfl_xor_sync(~0u, f, o);
    const int32_t mine = blockIdx.x * 32 + warp;
    if (lane == 0 && mine < C) dw[mine] = f;
}

// How rows are dealt to teams.
struct norm_shape {
    int32_t vpt, lanes, warps, threads, rows;           // rows: of a block and round
    int64_t blocks;
};

// vecs: vectors of a lane at most, as long as eight warps hold a row; inputs: of a row in shared memory, twice; busy: threads that an
// SM is to have.  Measured (bf16, 400 million values, floors 177, 412 and 236 us): best are four to six vectors a lane and one row
// ahead, 384 threads for a norm into 8 bits with a residual (2992 channels 406 us, 4096 443, 768 406; one warp of eight vectors, two rows
// ahead and 256 threads take 490 to 670) or with y (2048 channels 272 us for 170 million values; 512 threads 275), 512 into 8 bits alone (2048
// channels 264 us for 346 million values; 384 threads 300) and without 8 bits (236 to 253), 768 for rows into 8 bits (174 to 190; eight vectors and 256
// threads up to 390), 512 in the gradient; large blocks before small ones.
norm_shape norm_deal(int64_t rows, int32_t nv, int32_t vecs, int32_t inputs, int32_t busy, bool grad = false)
{
    norm_shape s;
    if (rows <= 2 * kSMs) vecs = 2;         // few rows take more lanes each
    s.lanes = 1;
    // narrow rows: four vectors a lane, not one (1 million rows of 128 bf16: quantised in 63 us for 98, the gradient 153 for 178)
    while (s.lanes < 32 && nv > s.lanes * std::min(vecs, 4)) s.lanes *= 2;
    s.warps = s.lanes < 32 ? 1 : std::min(kNormWarps, (nv + 32 * vecs - 1) / (32 * vecs));
    s.lanes *= s.warps;
    s.vpt = (nv + s.lanes - 1) / s.lanes;
    if (s.vpt == 7) s.vpt = 8;
    // rows of a block: whole warps, and blocks for all SMs
    const int32_t bytes = inputs * 2 * 16 * s.vpt * s.lanes, least = std::max(1, 32 / s.lanes);
    const int32_t most = std::max(1, std::min({std::min(busy, norm_threads(s.vpt, grad)) / s.lanes, kNormSmem / bytes}));
    s.rows = (int32_t)std::min<int64_t>(most, std::max<int64_t>(rows / kSMs, 1));
    s.rows = std::max(least, s.rows / least * least);
    s.threads = s.rows * s.lanes;
    const int32_t sm = std::max(1, std::min((busy + s.threads / 2) / s.threads, kNormSmem / (bytes * s.rows)));
    s.blocks = std::min<int64_t>((rows + s.rows - 1) / s.rows, kSMs * sm);
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

template <int BF16, int VPT, int NORM, int Q8, int RES>
cudaError_t norm_launch(const norm_shape &sh, const norm_args &a, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    auto *kernel = tdp_rms_norm_kernel<BF16, VPT, NORM, Q8, RES>;
    const cudaError_t e = tdp_allow_smem(kernel, kNormSmem, done);
    return e != cudaSuccess ? e : tdp_launch_smem(true, kernel, (unsigned)sh.blocks, sh.threads, (size_t)32 * (1 + RES) * VPT * sh.threads, s, a);
}

// Any row as one of eight vectors a lane (norm_deal's for 256 threads).
template <int RES>
cudaError_t norm_launch_small(int bf16, const norm_shape &sh, const norm_args &a, cudaStream_t s)
{
    return bf16 ? norm_launch<1, 8, 1, kSmall8, RES>(sh, a, s) : norm_launch<0, 8, 1, kSmall8, RES>(sh, a, s);
}

template <int NORM, int Q8, int RES>
cudaError_t norm_launch(int bf16, const norm_shape &sh, const norm_args &a, cudaStream_t s)
{
#define TDP_NORM(V) (bf16 ? norm_launch<1, V, NORM, Q8, RES>(sh, a, s) : norm_launch<0, V, NORM, Q8, RES>(sh, a, s))
    switch (sh.vpt) {
    case 1: return TDP_NORM(1);
    case 2: return TDP_NORM(2);
    case 3: return TDP_NORM(3);
    case 4: return TDP_NORM(4);
    case 5: return TDP_NORM(5);
    case 6: return TDP_NORM(6);
    default: return TDP_NORM(8);
    }
#undef TDP_NORM
}

template <int BF16, int VPT, int KEPT8>
cudaError_t grad_launch(const norm_shape &sh, const norm_grad_args &a, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    auto *kernel = tdp_rms_norm_grad_kernel<BF16, VPT, KEPT8>;
    const cudaError_t e = tdp_allow_smem(kernel, kNormSmem, done);
    return e != cudaSuccess ? e : tdp_launch_smem(true, kernel, (unsigned)sh.blocks, sh.threads, (size_t)96 * VPT * sh.threads, s, a);
}

template <int BF16, int KEPT8>
cudaError_t grad_launch(const norm_shape &sh, const norm_grad_args &a, cudaStream_t s)
{
    switch (sh.vpt) {
    case 1: return grad_launch<BF16, 1, KEPT8>(sh, a, s);
    case 2: return grad_launch<BF16, 2, KEPT8>(sh, a, s);
    case 3: return grad_launch<BF16, 3, KEPT8>(sh, a, s);
    case 4: return grad_launch<BF16, 4, KEPT8>(sh, a, s);
    case 5: return grad_launch<BF16, 5, KEPT8>(sh, a, s);
    case 6: return grad_launch<BF16, 6, KEPT8>(sh, a, s);
    default: return grad_launch<BF16, 8, KEPT8>(sh, a, s);
    }
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
    const int64_t n = rows * C * plan->g.esize, n8 = rows * C, nr = rows * 4;
    if (tdp_overlap(h, n, y, n) || tdp_overlap(y8, n8, x8, n8) || tdp_overlap(rstd, nr, y8_scale, nr) || tdp_overlap(rstd, nr, x8_scale, nr) ||
        tdp_overlap(y8_scale, nr, x8_scale, nr))
        return tdp_fail(TDP_ERR_INVALID_ARG, "two outputs in one buffer");
    for (const void *p : {x, res, static_cast<const void *>(h), static_cast<const void *>(y)})
        if (tdp_overlap(y8, n8, p, n) || tdp_overlap(x8, n8, p, n)) return tdp_fail(TDP_ERR_INVALID_ARG, "8-bit rows over others");
    if (tdp_partly(h, x, n) || tdp_partly(h, res, n) || tdp_partly(y, x, n) || tdp_partly(y, res, n))
        return tdp_fail(TDP_ERR_INVALID_ARG, "h or y over a part of x or res");
    const bool small = (y8 || x8) && eps < 0x1p-36f;
    const norm_shape sh = norm_deal(rows, nv, kNormVecs, res ? 2 : 1, small ? 256 : (y8 || x8) && (res || y) ? 384 : 512);
    norm_args a = {rows, C, nv, sh.lanes, sh.warps, eps, 1.f / (float)C, x, res, w, h, y, rstd, y8, x8, y8_scale, x8_scale};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int bf16 = plan->g.dtype == TDP_BF16;
    const cudaError_t err = small  ? (res ? norm_launch_small<1>(bf16, sh, a, s) : norm_launch_small<0>(bf16, sh, a, s))
                            : y8   ? (res ? norm_launch<1, kAny8, 1>(bf16, sh, a, s) : norm_launch<1, kAny8, 0>(bf16, sh, a, s))
                            : x8   ? (res ? norm_launch<1, kKept8, 1>(bf16, sh, a, s) : norm_launch<1, kKept8, 0>(bf16, sh, a, s))
                                   : (res ? norm_launch<1, kPlain, 1>(bf16, sh, a, s) : norm_launch<1, kPlain, 0>(bf16, sh, a, s));
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
    if (tdp_overlap(x8, rows * C, x, rows * C * plan->g.esize)) return tdp_fail(TDP_ERR_INVALID_ARG, "8-bit rows over x");
    const norm_shape sh = norm_deal(rows, nv, kNormVecs, 1, 768);
    norm_args a = {};
    a.rows = rows;
    a.C = C;
    a.nv = nv;
    a.lanes = sh.lanes;
    a.warps = sh.warps;
    a.x = x;
    a.x8 = x8;
    a.x8_scale = x8_scale;
    const cudaError_t err = norm_launch<0, kKept8, 0>(plan->g.dtype == TDP_BF16, sh, a, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}

extern "C" tdp_status tdp_rms_norm_grad_workspace(tdp_plan_t plan, int64_t rows, int32_t C, int64_t *bytes)
{
    int32_t nv = 0;
    if (!bytes) return tdp_fail(TDP_ERR_INVALID_ARG, "null bytes");
    const tdp_status st = norm_check(plan, rows, C, &nv);
    if (st != TDP_OK) return st;
    *bytes = norm_deal(rows, nv, kGradVecs, 3, 512, true).blocks * C * 4;
    return tdp_ok();
}

extern "C" tdp_status tdp_rms_norm_grad(tdp_plan_t plan, int64_t rows, int32_t C, const void *h, const uint8_t *x8,
                                        const float *x8_scale, const float *rstd, const void *w, const void *dy,
                                        const void *dh, void *dx, float *dw, void *ws, int64_t ws_bytes, tdp_stream_t stream)
{
    int32_t nv = 0;
    const tdp_status st = norm_check(plan, rows, C, &nv);
    if (st != TDP_OK) return st;
    const norm_shape sh = norm_deal(rows, nv, kGradVecs, 3, 512, true);
    if (rows > 0) {
        if (!rstd || !dy || !dx) return tdp_fail(TDP_ERR_INVALID_ARG, "null rstd, dy or dx");
        if (!h == !x8 || !x8 != !x8_scale) return tdp_fail(TDP_ERR_INVALID_ARG, "need h, or x8 with its scales, and not both");
        if (dw && (!ws || ws_bytes < sh.blocks * C * 4)) return tdp_fail(TDP_ERR_INVALID_ARG, "ws too small");
        if (!tdp_aligned(h, 16) || !tdp_aligned(x8, 16) || !tdp_aligned(w, 16) || !tdp_aligned(dy, 16) || !tdp_aligned(dh, 16) ||
            !tdp_aligned(dx, 16) || !tdp_aligned(x8_scale, 4) || !tdp_aligned(rstd, 4) || !tdp_aligned(ws, 256))
            return tdp_fail(TDP_ERR_MISALIGNED, "rows and w need 16-byte, scales and rstd 4-byte, ws 256-byte alignment");
        const int64_t n = rows * C * plan->g.esize;
        if (tdp_overlap(dx, n, x8, rows * C) || tdp_partly(dx, h, n) || tdp_partly(dx, dy, n) || tdp_partly(dx, dh, n))
            return tdp_fail(TDP_ERR_INVALID_ARG, "dx over x8, or a part of h, dy or dh");
    }
    if (!tdp_aligned(dw, 4)) return tdp_fail(TDP_ERR_MISALIGNED, "dw needs 4-byte alignment");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (rows > 0) {
        norm_grad_args a = {rows, C, nv, sh.lanes, sh.warps, 1.f / (float)C, h, w, dy, dh, x8, x8_scale, rstd, dx, dw ? static_cast<float *>(ws) : nullptr};
        err = plan->g.dtype == TDP_BF16 ? (x8 ? grad_launch<1, 1>(sh, a, s) : grad_launch<1, 0>(sh, a, s))
                                        : (x8 ? grad_launch<0, 1>(sh, a, s) : grad_launch<0, 0>(sh, a, s));
    }
    if (err == cudaSuccess && dw)
        err = tdp_launch(true, tdp_rms_norm_dw_kernel, (unsigned)((C + 31) / 32), 1024, s, static_cast<const float *>(ws), (int32_t)sh.blocks, C, dw);
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}
