// tdp_gnorm.cu -- group normalisation of every (tile, item), channels last, with an
// activation, and its gradients.
//
// Over the n = T_t * C/groups values of a group: mean, rstd = 1/sqrt(var + eps),
// z = (x - mean) * rstd * gamma + beta, y = act(z).  With h = (x - mean) * rstd,
// dz = dy * act'(z) and g = dz * gamma the gradient is
//   dx = rstd * (g - mean(g) - h * mean(g * h)),  dgamma = sum dz * h,  dbeta = sum dz.
//
// Bound by memory.  Two ways, by size:
//   - tdp_gn_sums_kernel, tdp_gn_apply_kernel: sums of chunks of rows, then the elementwise pass, whose blocks join
//     their segment's chunks themselves and run through the rows backwards, so that what the sums
//     read last is found in the 129 MB L2.  Rows come by way of shared memory, some 150 KB an SM on their way: loads into
//     registers, a batch after the other, took 601 us where this takes 570 (635 million bf16 values, 6.7 TB/s over the
//     three times that they move), and 1075 us in the gradient where this takes 984.  Tried: segments kept in the shared
//     memory of a cluster, read once in one launch: 97 us where this takes 35 (256 segments of 128 KB), 21 where this
//     takes 13 (one of 256 KB), in a graph 7.8 where this takes 5.5 (four of 4 KB): what it saves comes from L2 anyway
//     and its barriers cost more (the launch that it saves costs a host that launches one by one 4 us).  One grid
//     that takes chunks of sums and, some segments later, of the elementwise pass in turn: its tickets, joins and
//     flags took 934 us.  Slices of a few channels kept in a cluster read 32-byte pieces of rows, 2171 us.
//     Rows of more vectors than a block's 256 threads are split into slabs of whole groups (92 MB of 1280
//     channels, the gradient: 93 us against 344 in the way below).
//   - groups wider than 256 vectors: sums, join and elementwise pass as launches of their own.
// Variances are sums of squared deviations, of a block's values about their mean or joined by
// T. Chan's rule, so that a mean far from zero costs no digits.  Every join runs in a fixed order.
#include <algorithm>
#include <atomic>
#include <numeric>

#include "tdp.h"
#include "tdp_internal.h"
#include "tdp_rows.cuh"

namespace {

constexpr int kGnThreads = 256;
constexpr int kGnWideRows = 256;            // rows of a chunk at most, groups wider than a block
constexpr int kGnBlocks = 3;                // blocks that an SM holds
constexpr int kGnChunkMost = 256 << 10;     // bytes of x of a chunk: 128 KB 620 us, 350 KB 575 us where this takes 570
constexpr int kGnChunkLeast = 32 << 10;

// SiLU is z * s, s = 1 / (1 + exp(-z)); its slope s + z s (1 - s).  exp(-z) overflows to infinity for z below -88: s = 0,
// SiLU's limit.  The gradient kernels are bound by instructions as much as by memory: two table instructions and a
// dozen others an element.
__device__ __forceinline__ float sigmoidf(float z)
{
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    return s;
}
template <int ACT>
__device__ __forceinline__ float act(float z) { return ACT ? z * sigmoidf(z) : z; }
template <int ACT>
__device__ __forceinline__ float act_grad(float z)
{
    if (!ACT) return 1.f;
    const float s = sigmoidf(z), t = z * s;
    return fmaf(-t, s, t) + s;
}

struct gn_args {
    int32_t C, G, cg;           // channels, groups, channels per group
    fast_div by_cg;
    int32_t chunks, rows;       // chunks per segment, rows per chunk
    uint32_t pblocks;           // blocks that add up dgamma and dbeta
    int32_t slabs, slab;        // blocks side by side on a row, channels of each: whole groups
    float eps;
    const void *x, *gamma, *beta, *dy;
    void *y;                    // y or dx
    float *mean, *rstd;         // [segments, G]
    float *dgamma, *dbeta;      // [C]
    float *part;                // sums of chunks per channel [segments, chunks, C, 2]
    float *gpart;               // ... per group [segments, chunks, G, 2]
    float *coef;                // wide, gradient: a segment's sums [segments, C, 2]
    float *gmean;               // wide, gradient: means of g and g * h [segments, G, 2]
};

// A thread's vector of channels: 16 bytes, 8 bytes of bf16 in the gradient (its seven constants a channel leave
// registers for four channels).
template <int BF16, int GRAD>
struct gn_vec {
    static constexpr int V = BF16 && !GRAD ? 8 : 4;
    using type = uint4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *f) { tdp_elem<BF16>::unpack(u, f); }
    static __device__ __forceinline__ uint4 pack(const float *f) { return tdp_elem<BF16>::pack(f); }
};
template <>
struct gn_vec<1, 1> {
    static constexpr int V = 4;
    using type = uint2;
    static __device__ __forceinline__ void unpack(const uint2 &u, float *f)
    {
        f[0] = tdp_bf16_lo(u.x);
        f[1] = tdp_bf16_hi(u.x);
        f[2] = tdp_bf16_lo(u.y);
        f[3] = tdp_bf16_hi(u.y);
    }
    static __device__ __forceinline__ uint2 pack(const float *f) { return make_uint2(tdp_pack_bf16x2(f[0], f[1]), tdp_pack_bf16x2(f[2], f[3])); }
};
constexpr int gn_width(int bf16, int grad) { return bf16 && !grad ? 8 : 4; }

template <int BF16>
__device__ __forceinline__ float param(const void *p, int32_t c, float none)
{
    using T = typename tdp_elem<BF16>::type;
    return p ? (float)static_cast<const T *>(p)[c] : none;
}

// A thread's column of V channels and their constants.
template <int BF16, int GRAD>
struct gn_cols {
    using E = gn_vec<BF16, GRAD>;
    static constexpr int V = E::V;
    float mu[V], a[V], b[V];        // z = (x - mu) * a + b
    float rs[V], ga[V], m1[V], m2[V];
    __device__ __forceinline__ void params(const gn_args &g, int32_t col)
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            ga[j] = 1.f;
            b[j] = 0.f;
        }
        // plain loads: the kernel before, which may have written them, can overlap this one
        if (g.gamma) E::unpack(static_cast<const typename E::type *>(g.gamma)[col], ga);
        if (g.beta) E::unpack(static_cast<const typename E::type *>(g.beta)[col], b);
    }
    __device__ __forceinline__ void moments(const gn_args &g, int64_t s, int32_t col)
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t gr = s * g.G + g.by_cg.div(col * V + j);
            mu[j] = __ldcg(g.mean + gr);
            rs[j] = __ldcg(g.rstd + gr);
        }
        params(g, col);
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = rs[j] * ga[j];
    }
    __device__ __forceinline__ void means(const gn_args &g, int64_t s, int32_t col)
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t gr = s * g.G + g.by_cg.div(col * V + j);
            m1[j] = __ldcg(g.gmean + 2 * gr) * rs[j];
            m2[j] = __ldcg(g.gmean + 2 * gr + 1) * rs[j];
        }
    }
    template <int ACT>
    __device__ __forceinline__ void forward(float *f) const
    {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = act<ACT>((f[j] - mu[j]) * a[j] + b[j]);
    }
    // dz and h of one row
    template <int ACT>
    __device__ __forceinline__ void grad(const float *x, const float *dy, int j, float &dz, float &h) const
    {
        h = (x[j] - mu[j]) * rs[j];
        dz = dy[j] * act_grad<ACT>(h * ga[j] + b[j]);
    }
    template <int ACT>
    __device__ __forceinline__ void backward(const float *x, float *dy) const
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float dz, h;
            grad<ACT>(x, dy, j, dz, h);
            dy[j] = fmaf(dz, a[j], -fmaf(h, m2[j], m1[j]));        // a = rstd * gamma, m1 and m2 times rstd
        }
    }
};

// Sum over `width` neighbouring lanes (a power of two).
__device__ __forceinline__ float lanes_sum(float x, int32_t width = 32)
{
    for (int o = width / 2; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

// Threads of a block on groups: as many lanes a group as let all groups be joined at once, where there are few; a
// warp each took four turns of dependent loads and shuffles at 32 groups, 3 us a block.  f(group, on) runs in
// whole warps, past the last group too (on = false).
struct gn_team {
    int32_t width, lane, first, step;
    __device__ __forceinline__ gn_team(int32_t G, int32_t threads)
    {
        width = 32;
        while (width > 1 && threads / width < G) width >>= 1;
        lane = threadIdx.x & (width - 1);
        first = threadIdx.x / width;
        step = threads / width;
    }
    template <typename F>
    __device__ __forceinline__ void each(int32_t G, F f) const
    {
        for (int32_t g0 = 0; g0 < G; g0 += step) f(g0 + first, g0 + first < G);
    }
};

// Moments of a group from parts (mean m_i, squared deviations q_i, n_i values each) by `width` lanes; value i by at(i).
// The mean is summed from the first part's on: weighted means themselves would leave roundings of the mean's own size, a
// spread where a group holds one value over and over.
template <typename At>
__device__ __forceinline__ void join_moments(int32_t parts, int32_t lane, int32_t width, float n, At at, float &mean, float &q)
{
    const float first = parts > 0 ? at(0).x : 0.f;
    mean = 0.f;
    for (int32_t i = lane; i < parts; i += width) {
        const float3 p = at(i);
        mean += (p.x - first) * (p.z / n);
    }
    mean = first + lanes_sum(mean, width);
    q = 0.f;
    for (int32_t i = lane; i < parts; i += width) {
        const float3 p = at(i);
        q += p.y + p.z * (p.x - mean) * (p.x - mean);
    }
    q = lanes_sum(q, width);
}

// Threads of a block on rows of CV <= kThreads vectors: `step` rows side by side.
struct gn_lane {
    int32_t col, row, step, w;
    bool on;
    __device__ __forceinline__ gn_lane(int32_t CV, int32_t threads)
    {
        w = CV;
        step = threads / w;
        row = threadIdx.x / w;
        col = threadIdx.x - row * w;
        on = row < step;
    }
};

// ------------------------------------------------------------------ two passes
// A thread's vectors of x (and dy) by way of shared memory, kDeep - 1 groups of kGroup rows on their way at any time:
// copied, and waited for, by the thread that uses them, so that no thread waits for another.
template <int BF16, int GRAD>
struct gn_feed {
    using X = typename gn_vec<BF16, GRAD>::type;
    static constexpr int kGroup = GRAD && !BF16 ? 2 : 4, kDeep = GRAD ? 3 : 4;
    static constexpr int kBytes = kDeep * kGroup * kGnThreads * (int)sizeof(X) * (GRAD ? 2 : 1);
    static_assert(kBytes >= kGnThreads * (gn_vec<BF16, GRAD>::V * 8 + 4), "the sums' join takes the same memory");
    uint32_t at;
    const X *x, *dy;
    int32_t step, left, put = 0, get = 0;       // elements between rows; rows still to be asked for; stages
    __device__ __forceinline__ gn_feed(void *smem, const X *x0, const X *dy0, int32_t step_, int32_t rows)
        : at((uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * (int)sizeof(X)), x(x0), dy(dy0), step(step_), left(rows)
    {
#pragma unroll
        for (int i = 0; i < kDeep - 1; ++i) ask();
    }
    static __device__ __forceinline__ void copy(uint32_t to, const X *from)
    {
        if (sizeof(X) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
    }
    __device__ __forceinline__ uint32_t slot(int32_t stage, int v, int which) const
    {
        return at + ((stage * kGroup + v) * (GRAD ? 2 : 1) + which) * (kGnThreads * (int)sizeof(X));
    }
    __device__ __forceinline__ void ask()
    {
#pragma unroll
        for (int v = 0; v < kGroup; ++v)
            if (v < left) {
                copy(slot(put, v, 0), x);
                x += step;
                if (GRAD) {
                    copy(slot(put, v, 1), dy);
                    dy += step;
                }
            }
        left -= kGroup;
        put = put + 1 == kDeep ? 0 : put + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    static __device__ __forceinline__ X read(uint32_t from)
    {
        X v;
        if constexpr (sizeof(X) == 16)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
        else
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(from) : "memory");
        return v;
    }
    // the next group, its stage's successor asked for
    __device__ __forceinline__ void next(X *u, X *d)
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 2) : "memory");
#pragma unroll
        for (int v = 0; v < kGroup; ++v) {
            u[v] = read(slot(get, v, 0));
            if (GRAD) d[v] = read(slot(get, v, 1));
        }
        get = get + 1 == kDeep ? 0 : get + 1;
        ask();
    }
};

// Adds up (GRAD) or joins by Chan's rule the row lanes' values (s1, s2) of each channel; red holds threads * V
// pairs, then a count per thread.  Afterwards row lane 0's entries are the block's.  n: this thread's rows.
template <int V, int GRAD>
__device__ __forceinline__ void join_lanes(float2 *red, const gn_lane &l, float n, const float *s1, const float *s2)
{
    float2 *mine = red + threadIdx.x * V;
    float *count = reinterpret_cast<float *>(red + kGnThreads * V) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < V; ++j) mine[j] = make_float2(s1[j], s2[j]);
    *count = n;
    __syncthreads();
    for (int32_t live = l.step; live > 1;) {
        const int32_t half = (live + 1) / 2;
        if (l.on && l.row + half < live) {
            const float2 *o = mine + half * l.w * V;
            if (GRAD) {
#pragma unroll
                for (int j = 0; j < V; ++j) mine[j] = make_float2(mine[j].x + o[j].x, mine[j].y + o[j].y);
            } else {
                const float na = *count, nb = count[half * l.w];
                if (nb > 0.f) {
                    const float wb = nb / (na + nb);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float d = o[j].x - mine[j].x;
                        mine[j] = make_float2(mine[j].x + d * wb, mine[j].y + o[j].y + d * d * na * wb);
                    }
                    *count = na + nb;
                }
            }
        }
        __syncthreads();
        live = half;
    }
}

// Sums of one chunk of a segment: per group (gradient: of g and g * h, and per channel of dz and dz * h).
template <int BF16, int GRAD, int ACT>
__global__ void __launch_bounds__(kGnThreads, kGnBlocks)
tdp_gn_sums_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    using E = gn_vec<BF16, GRAD>;
    using X = typename E::type;
    constexpr int V = E::V;
    extern __shared__ __align__(16) unsigned char dyn[];
    float2 *red = reinterpret_cast<float2 *>(dyn);      // after the last rows: [threads * V + threads / 2]
    const int32_t unit = blockIdx.x / a.slabs, s = unit / a.chunks, ch = unit % a.chunks, CV = a.C / V;
    const int32_t c0 = (blockIdx.x - unit * a.slabs) * a.slab, cs = min(a.slab, a.C - c0), G0 = c0 / a.cg, Gs = cs / a.cg;      // slab
    const tdp_seg seg = tdp_seg_at(g, s);
    const int64_t r0 = (int64_t)ch * a.rows;
    const int32_t rows = (int32_t)min((int64_t)a.rows, seg.T - r0);
    const gn_lane l(cs / V, kGnThreads);
    float2 *chan = reinterpret_cast<float2 *>(a.part) + (int64_t)unit * a.C + c0;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    if (rows <= 0) {
        // a shorter segment: its parts of dgamma and dbeta are nothing
        if (GRAD && a.dgamma)
            for (int32_t c = threadIdx.x; c < cs; c += kGnThreads) chan[c] = make_float2(0.f, 0.f);
        return;
    }
    float p[V], s1[V], s2[V], n = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = s1[j] = s2[j] = 0.f;
    if (l.on && l.row < rows) {
        const int32_t col = c0 / V + l.col;
        const X *x = reinterpret_cast<const X *>(a.x) + (seg.row0 + r0) * CV + col;
        const X *dy = reinterpret_cast<const X *>(a.dy) + (seg.row0 + r0) * CV + col;
        gn_cols<BF16, GRAD> k;
        const int32_t mine = (rows - l.row + l.step - 1) / l.step, step = l.step * CV;     // rows of this thread
        auto add = [&](const X &xv, const X &dv) {
            float f[V], e[V];
            E::unpack(xv, f);
            if (GRAD) E::unpack(dv, e);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (GRAD) {
                    float dz, h;
                    k.template grad<ACT>(f, e, j, dz, h);
                    s1[j] += dz;
                    s2[j] = fmaf(dz, h, s2[j]);
                } else {
                    const float t = f[j] - p[j];
                    s1[j] += t;
                    s2[j] = fmaf(t, t, s2[j]);
                }
            }
        };
        gn_feed<BF16, GRAD> feed(dyn, x + l.row * CV, dy + l.row * CV, step, mine);
        if (GRAD) k.moments(a, s, col);
        constexpr int U = feed.kGroup;
        for (int32_t i = 0; i < mine; i += U) {
            X u[U], d[U];
            feed.next(u, d);
            if (!GRAD && i == 0) E::unpack(u[0], p);            // deviations from the thread's own first value
#pragma unroll
            for (int v = 0; v < U; ++v)
                if (i + v < mine) add(u[v], d[v]);
        }
        if (!GRAD) {
            n = (float)mine;
            const float inv = 1.f / n;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float m = s1[j] * inv;
                s2[j] -= s1[j] * m;             // squared deviations from the thread's mean
                s1[j] = p[j] + m;
            }
        }
    }
    __syncthreads();
    join_lanes<V, GRAD>(red, l, n, s1, s2);
    float2 *out = reinterpret_cast<float2 *>(a.gpart) + (int64_t)unit * a.G + G0;
    if (GRAD && a.dgamma)
        for (int32_t c = threadIdx.x; c < cs; c += kGnThreads) chan[c] = red[c];
    const gn_team team(Gs, kGnThreads);
    team.each(Gs, [&](int32_t gr, bool on) {
        float m = 0.f, q = 0.f;
        const int32_t many = on ? a.cg : 0;
        if (GRAD) {
            for (int32_t i = team.lane; i < many; i += team.width) {
                const float2 v = red[gr * a.cg + i];
                const float w = param<BF16>(a.gamma, c0 + gr * a.cg + i, 1.f);
                m += v.x * w;
                q += v.y * w;
            }
            m = lanes_sum(m, team.width);
            q = lanes_sum(q, team.width);
        } else {
            join_moments(many, team.lane, team.width, (float)a.cg * rows, [&](int32_t i) {
                const float2 v = red[gr * a.cg + i];
                return make_float3(v.x, v.y, (float)rows);
            }, m, q);
        }
        if (on && team.lane == 0) out[gr] = make_float2(m, q);
    });
}

// dgamma and dbeta from `parts` sums per channel: a block per four channels (a sector of each part), 64 threads a
// channel, their sums added in order.  red: kGnThreads pairs.
__device__ __forceinline__ void gn_params(const gn_args &a, const float2 *part, int32_t parts, int32_t block, float2 *red)
{
    const int32_t c = block * 4 + (threadIdx.x & 3);
    float2 t = make_float2(0.f, 0.f);
    if (c < a.C)
#pragma unroll 8
        for (int32_t i = threadIdx.x >> 2; i < parts; i += kGnThreads / 4) {
            const float2 v = part[(int64_t)i * a.C + c];
            t.x += v.x;
            t.y += v.y;
        }
    red[threadIdx.x] = t;
    for (int k = kGnThreads / 2; k >= 4; k /= 2) {
        __syncthreads();
        if (threadIdx.x < k) {
            red[threadIdx.x].x += red[threadIdx.x + k].x;
            red[threadIdx.x].y += red[threadIdx.x + k].y;
        }
    }
    if (threadIdx.x >= 4 || c >= a.C) return;
    a.dbeta[c] = red[threadIdx.x].x;
    a.dgamma[c] = red[threadIdx.x].y;
}

// The elementwise pass of one chunk, chunks from the last to the first; the block joins its segment's sums.  In the
// gradient the first a.pblocks blocks add up dgamma and dbeta under it (a launch of their own took 7 us).
template <int BF16, int GRAD, int ACT>
__global__ void __launch_bounds__(kGnThreads, kGnBlocks)
tdp_gn_apply_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    using E = gn_vec<BF16, GRAD>;
    using X = typename E::type;
    constexpr int V = E::V;
    extern __shared__ __align__(16) unsigned char dyn[];
    float2 *grp = reinterpret_cast<float2 *>(dyn + gn_feed<BF16, GRAD>::kBytes);             // [G]
    if (GRAD && blockIdx.x < a.pblocks) {
        tdp_pdl_trigger();
        tdp_pdl_wait();
        gn_params(a, reinterpret_cast<const float2 *>(a.part), (int32_t)((gridDim.x - a.pblocks) / a.slabs), blockIdx.x, reinterpret_cast<float2 *>(dyn));
        return;
    }
    const int32_t at_unit = gridDim.x - 1 - blockIdx.x, unit = at_unit / a.slabs, s = unit / a.chunks, ch = unit % a.chunks, CV = a.C / V;
    const int32_t c0 = (at_unit - unit * a.slabs) * a.slab, cs = min(a.slab, a.C - c0), G0 = c0 / a.cg, Gs = cs / a.cg;      // slab
    const tdp_seg seg = tdp_seg_at(g, s);
    const int64_t r0 = (int64_t)ch * a.rows;
    const int32_t rows = (int32_t)min((int64_t)a.rows, seg.T - r0), chunks = (int32_t)((seg.T + a.rows - 1) / a.rows);
    const gn_lane l(cs / V, kGnThreads);
    const int32_t col = c0 / V + l.col;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    if (rows <= 0) return;
    const int64_t at = (seg.row0 + r0) * CV + col;
    const X *x = reinterpret_cast<const X *>(a.x) + at, *dy = reinterpret_cast<const X *>(a.dy) + at;
    X *y = reinterpret_cast<X *>(a.y) + at;
    const int32_t mine = l.on ? (rows - l.row + l.step - 1) / l.step : 0, step = l.step * CV;        // rows of this thread
    gn_feed<BF16, GRAD> feed(dyn, x + l.row * CV, dy + l.row * CV, step, mine);         // ahead of the join
    const float n = (float)seg.T * a.cg;
    const float2 *part = reinterpret_cast<const float2 *>(a.gpart) + (int64_t)s * a.chunks * a.G + G0;
    const gn_team team(Gs, kGnThreads);
    team.each(Gs, [&](int32_t gr, bool on) {
        float m = 0.f, q = 0.f;
        const int32_t many = on ? chunks : 0;
        if (GRAD) {
#pragma unroll 4
            for (int32_t i = team.lane; i < many; i += team.width) {
                const float2 v = part[(int64_t)i * a.G + gr];
                m += v.x;
                q += v.y;
            }
            m = lanes_sum(m, team.width) / n;
            q = lanes_sum(q, team.width) / n;
        } else {
            join_moments(many, team.lane, team.width, n, [&](int32_t i) {
                const float2 v = part[(int64_t)i * a.G + gr];
                return make_float3(v.x, v.y, (float)min((int64_t)a.rows, seg.T - (int64_t)i * a.rows) * a.cg);
            }, m, q);
            q = 1.f / sqrtf(q / n + a.eps);
            if (on && ch == 0 && team.lane == 0) {
                a.mean[(int64_t)s * a.G + G0 + gr] = m;
                a.rstd[(int64_t)s * a.G + G0 + gr] = q;
            }
        }
        if (on && team.lane == 0) grp[gr] = make_float2(m, q);
    });
    __syncthreads();
    if (!l.on || l.row >= rows) return;
    gn_cols<BF16, GRAD> k;
    if (GRAD) k.moments(a, s, col);
    else k.params(a, col);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float2 v = grp[a.by_cg.div(l.col * V + j)];
        if (GRAD) {
            k.m1[j] = v.x * k.rs[j];
            k.m2[j] = v.y * k.rs[j];
        } else {
            k.mu[j] = v.x;
            k.a[j] = v.y * k.ga[j];
        }
    }
    auto put = [&](const X &xv, const X &dv, int32_t o) {
        float f[V], e[V];
        E::unpack(xv, f);
        if (GRAD) {
            E::unpack(dv, e);
            k.template backward<ACT>(f, e);
            __stcs(y + o, E::pack(e));
        } else {
            k.template forward<ACT>(f);
            __stcs(y + o, E::pack(f));
        }
    };
    constexpr int U = feed.kGroup;
    for (int32_t i = 0, off = l.row * CV; i < mine; i += U) {
        X u[U], d[U];
        feed.next(u, d);
#pragma unroll
        for (int v = 0; v < U; ++v, off += step)
            if (i + v < mine) put(u[v], d[v], off);
    }
}

// ------------------------------------------------------------------ wide groups
// A thread per column of vectors; blockIdx.y takes 256 of them.
template <int BF16, int GRAD, int ACT>
__global__ void __launch_bounds__(kGnThreads)
tdp_gn_wide_sums_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    using E = gn_vec<BF16, GRAD>;
    using X = typename E::type;
    constexpr int V = E::V;
    const int32_t s = blockIdx.x / a.chunks, ch = blockIdx.x % a.chunks, CV = a.C / V, col = blockIdx.y * kGnThreads + threadIdx.x;
    const tdp_seg seg = tdp_seg_at(g, s);
    const int64_t r0 = (int64_t)ch * a.rows;
    const int32_t rows = (int32_t)min((int64_t)a.rows, seg.T - r0);
    tdp_pdl_trigger();
    tdp_pdl_wait();
    if (rows <= 0 || col >= CV) return;
    const int64_t at = (seg.row0 + r0) * CV + col;
    const X *x = reinterpret_cast<const X *>(a.x) + at, *dy = reinterpret_cast<const X *>(a.dy) + at;
    float p[V], s1[V], s2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s1[j] = s2[j] = 0.f;
    E::unpack(x[0], p);
    gn_cols<BF16, GRAD> k;
    if (GRAD) k.moments(a, s, col);
#pragma unroll 4
    for (int32_t r = 0; r < rows; ++r) {
        float f[V], e[V];
        E::unpack(x[(int64_t)r * CV], f);
        if (GRAD) E::unpack(dy[(int64_t)r * CV], e);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (GRAD) {
                float dz, h;
                k.template grad<ACT>(f, e, j, dz, h);
                s1[j] += dz;
                s2[j] += dz * h;
            } else {
                const float t = f[j] - p[j];
                s1[j] += t;
                s2[j] += t * t;
            }
        }
    }
    float2 *out = reinterpret_cast<float2 *>(a.part) + ((int64_t)s * a.chunks + ch) * a.C + col * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float m = s1[j] / rows;
        out[j] = GRAD ? make_float2(s1[j], s2[j]) : make_float2(p[j] + m, s2[j] - s1[j] * m);
    }
}

// One warp per (segment, group): the group's moments, or (gradient) its channels' sums and means of g and g * h.
template <int BF16, int GRAD>
__global__ void __launch_bounds__(kGnThreads)
tdp_gn_wide_join_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const int64_t w = ((int64_t)blockIdx.x * kGnThreads + threadIdx.x) >> 5;
    const int32_t lane = threadIdx.x & 31;
    if (w >= (int64_t)g.nt * g.B * a.G) return;
    const int32_t s = (int32_t)(w / a.G), gr = (int32_t)(w % a.G);
    const tdp_seg seg = tdp_seg_at(g, s);
    const int32_t chunks = (int32_t)((seg.T + a.rows - 1) / a.rows);
    const float2 *part = reinterpret_cast<const float2 *>(a.part) + (int64_t)s * a.chunks * a.C + gr * a.cg;
    const float n = (float)seg.T * a.cg;
    if (!GRAD) {
        float m, q;
        join_moments(chunks * a.cg, lane, 32, n, [&](int32_t i) {
            const int32_t k = i / a.cg;
            const float2 v = part[(int64_t)k * a.C + i - k * a.cg];
            return make_float3(v.x, v.y, (float)min((int64_t)a.rows, seg.T - (int64_t)k * a.rows));
        }, m, q);
        if (lane == 0) {
            a.mean[w] = m;
            a.rstd[w] = 1.f / sqrtf(q / n + a.eps);
        }
    } else {
        float x = 0.f, y = 0.f;
        for (int32_t i = lane; i < a.cg; i += 32) {
            float2 t = make_float2(0.f, 0.f);
            for (int32_t k = 0; k < chunks; ++k) {
                const float2 v = part[(int64_t)k * a.C + i];
                t.x += v.x;
                t.y += v.y;
            }
            reinterpret_cast<float2 *>(a.coef)[(int64_t)s * a.C + gr * a.cg + i] = t;
            const float k = param<BF16>(a.gamma, gr * a.cg + i, 1.f);
            x += t.x * k;
            y += t.y * k;
        }
        x = lanes_sum(x);
        y = lanes_sum(y);
        if (lane == 0) {
            a.gmean[2 * w] = x / n;
            a.gmean[2 * w + 1] = y / n;
        }
    }
}

template <int BF16, int GRAD, int ACT>
__global__ void __launch_bounds__(kGnThreads)
tdp_gn_wide_apply_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    using E = gn_vec<BF16, GRAD>;
    using X = typename E::type;
    constexpr int V = E::V;
    const int32_t s = blockIdx.x / a.chunks, ch = blockIdx.x % a.chunks, CV = a.C / V, col = blockIdx.y * kGnThreads + threadIdx.x;
    const tdp_seg seg = tdp_seg_at(g, s);
    const int64_t r0 = (int64_t)ch * a.rows;
    const int32_t rows = (int32_t)min((int64_t)a.rows, seg.T - r0);
    tdp_pdl_trigger();
    tdp_pdl_wait();
    if (rows <= 0 || col >= CV) return;
    const int64_t at = (seg.row0 + r0) * CV + col;
    const X *x = reinterpret_cast<const X *>(a.x) + at, *dy = reinterpret_cast<const X *>(a.dy) + at;
    X *y = reinterpret_cast<X *>(a.y) + at;
    gn_cols<BF16, GRAD> k;
    k.moments(a, s, col);
    if (GRAD) k.means(a, s, col);
#pragma unroll 4
    for (int32_t r = 0; r < rows; ++r) {
        float f[V], e[V];
        E::unpack(x[(int64_t)r * CV], f);
        if (GRAD) {
            E::unpack(dy[(int64_t)r * CV], e);
            k.template backward<ACT>(f, e);
            y[(int64_t)r * CV] = E::pack(e);
        } else {
            k.template forward<ACT>(f);
            y[(int64_t)r * CV] = E::pack(f);
        }
    }
}

__global__ void __launch_bounds__(kGnThreads)
tdp_gn_wide_param_kernel(const gn_args a, int32_t segs)
{
    __shared__ float2 red[kGnThreads];
    tdp_pdl_trigger();
    tdp_pdl_wait();
    gn_params(a, reinterpret_cast<const float2 *>(a.coef), segs, blockIdx.x, red);
}

// ------------------------------------------------------------------ host
struct gn_plan {
    bool wide;
    int32_t chunks, rows, slabs, slab;
    int64_t gpart_at, coef_at, gmean_at, bytes;
};

tdp_status gn_check(tdp_plan_t plan, int32_t C, int32_t groups, int grad, gn_plan *p)
{
    if (!plan) return tdp_fail(TDP_ERR_INVALID_ARG, "null plan");
    const tdp_geom &g = plan->g;
    if (C < 1 || groups < 1 || C % groups != 0)
        return tdp_fail(TDP_ERR_INVALID_ARG, "need groups >= 1 dividing C");
    if (((int64_t)C * g.esize) % 16 != 0)
        return tdp_fail(TDP_ERR_MISALIGNED, "C * element size must be a multiple of 16 bytes");
    const int V = gn_width(g.dtype == TDP_BF16, grad);
    const int64_t CV = C / V, bytes = V * g.esize, T = tdp_max_tile_tokens(g), segs = (int64_t)g.nt * g.B;
    if (CV > (int64_t)kGnThreads * 65535 || (int64_t)g.B * g.total > ((int64_t)1 << 56) / C)
        return tdp_fail(TDP_ERR_TOO_LARGE, "group normalisation beyond index ranges");
    // rows of more vectors than a block has threads are split into slabs of whole groups and vectors
    const int64_t piece = std::lcm((int64_t)(C / groups), (int64_t)V), pieces = C / piece, fit = (int64_t)kGnThreads * V / piece;
    p->wide = fit == 0;
    p->slabs = p->wide ? 1 : (int32_t)((pieces + fit - 1) / fit);
    p->slab = (int32_t)((pieces + p->slabs - 1) / p->slabs * piece);
    if (p->wide) {
        // as many blocks as fill the device, of 16 rows at least
        const int64_t fill = (int64_t)g.B * g.total * ((CV + kGnThreads - 1) / kGnThreads) / (152 * 8);
        p->rows = (int32_t)std::min<int64_t>(std::max<int64_t>(fill, 16), kGnWideRows);
    } else {
        // chunks for whole rounds of the blocks that the device holds; a segment's last chunk is half full on average
        const int64_t all = (int64_t)g.B * g.total, round = 152 * kGnBlocks, most = round * kGnChunkMost;
        const int64_t units = (all * CV * bytes + most - 1) / most * round;
        const int64_t want = (all * p->slabs + units - 1) / std::max<int64_t>(units - segs * p->slabs / 2, 1);
        const int64_t row = (int64_t)p->slab * g.esize, least = (kGnChunkLeast + row - 1) / row;
        p->rows = (int32_t)std::max(std::min(want, T), least);
    }
    const int64_t chunks = (T + p->rows - 1) / p->rows;
    if (chunks * segs * p->slabs > 0x7fffffffLL - (C + 3) / 4) return tdp_fail(TDP_ERR_TOO_LARGE, "group normalisation beyond index ranges");
    p->chunks = (int32_t)chunks;
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    p->gpart_at = up(segs * p->chunks * C * 8);
    p->coef_at = p->gpart_at + up(segs * p->chunks * groups * 8);
    p->gmean_at = p->coef_at + up(segs * C * 8);
    p->bytes = p->gmean_at + up(segs * groups * 8);
    return TDP_OK;
}

template <typename K, typename... A>
cudaError_t gn_launch(K kernel, dim3 grid, size_t smem, cudaStream_t s, A... args)
{
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kGnThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int BF16, int GRAD, int ACT>
cudaError_t gn_run(const tdp_geom &g, const gn_plan &p, const gn_args &a, cudaStream_t s)
{
    const int64_t segs = (int64_t)g.nt * g.B;
    constexpr int V = gn_width(BF16, GRAD);
    cudaError_t err = cudaSuccess;
    auto blocks = [](int64_t threads) { return dim3((unsigned)((threads + kGnThreads - 1) / kGnThreads)); };
    if (!p.wide) {
        // the kernels' shared-memory limits, raised once per device
        static std::atomic<bool> done[64];
        constexpr int feed = gn_feed<BF16, GRAD>::kBytes;
        int dev = 0;
        err = cudaGetDevice(&dev);
        if (err == cudaSuccess && (dev >= 64 || !done[dev].load(std::memory_order_relaxed))) {
            const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
            err = cudaFuncSetAttribute(tdp_gn_sums_kernel<BF16, GRAD, ACT>, attr, feed);
            if (err == cudaSuccess) err = cudaFuncSetAttribute(tdp_gn_apply_kernel<BF16, GRAD, ACT>, attr, feed + kGnThreads * V * 8);
            if (err == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
        }
        const dim3 grid((unsigned)(segs * p.chunks * p.slabs));
        if (err == cudaSuccess) err = gn_launch(tdp_gn_sums_kernel<BF16, GRAD, ACT>, grid, (size_t)feed, s, g, a);
        if (err == cudaSuccess) err = gn_launch(tdp_gn_apply_kernel<BF16, GRAD, ACT>, dim3(grid.x + a.pblocks), (size_t)feed + a.slab / a.cg * 8, s, g, a);
    } else {
        const dim3 grid((unsigned)(segs * p.chunks), (unsigned)((a.C / V + kGnThreads - 1) / kGnThreads));
        err = gn_launch(tdp_gn_wide_sums_kernel<BF16, GRAD, ACT>, grid, 0, s, g, a);
        if (err == cudaSuccess) err = gn_launch(tdp_gn_wide_join_kernel<BF16, GRAD>, blocks(segs * a.G * 32), 0, s, g, a);
        if (err == cudaSuccess && GRAD && a.dgamma)
            err = gn_launch(tdp_gn_wide_param_kernel, dim3((unsigned)((a.C + 3) / 4)), 0, s, a, (int32_t)segs);
        if (err == cudaSuccess) err = gn_launch(tdp_gn_wide_apply_kernel<BF16, GRAD, ACT>, grid, 0, s, g, a);
    }
    return err;
}

template <int GRAD>
cudaError_t gn_dispatch(const tdp_geom &g, const gn_plan &p, gn_args a, int32_t act, void *ws, cudaStream_t s)
{
    unsigned char *w = static_cast<unsigned char *>(ws);
    a.cg = a.C / a.G;
    a.by_cg = fast_div_by(a.cg);
    a.chunks = p.chunks;
    a.rows = p.rows;
    a.slabs = p.slabs;
    a.slab = p.slab;
    a.pblocks = GRAD && a.dgamma ? (a.C + 3) / 4 : 0;
    a.part = reinterpret_cast<float *>(w);
    a.gpart = reinterpret_cast<float *>(w + p.gpart_at);
    a.coef = reinterpret_cast<float *>(w + p.coef_at);
    a.gmean = reinterpret_cast<float *>(w + p.gmean_at);
    if (g.dtype == TDP_BF16) return act ? gn_run<1, GRAD, 1>(g, p, a, s) : gn_run<1, GRAD, 0>(g, p, a, s);
    return act ? gn_run<0, GRAD, 1>(g, p, a, s) : gn_run<0, GRAD, 0>(g, p, a, s);
}

}  // namespace

extern "C" tdp_status tdp_group_norm_workspace(tdp_plan_t plan, int32_t C, int32_t groups, int64_t *bytes)
{
    gn_plan f, b;
    if (!bytes) return tdp_fail(TDP_ERR_INVALID_ARG, "null bytes");
    tdp_status st = gn_check(plan, C, groups, 0, &f);
    if (st == TDP_OK) st = gn_check(plan, C, groups, 1, &b);
    if (st != TDP_OK) return st;
    *bytes = std::max(f.bytes, b.bytes);
    return tdp_ok();
}

extern "C" tdp_status tdp_group_norm(tdp_plan_t plan, int32_t C, int32_t groups, float eps, int32_t act, const void *x,
                                     const void *gamma, const void *beta, void *y, float *mean, float *rstd, void *ws,
                                     int64_t ws_bytes, tdp_stream_t stream)
{
    gn_plan p;
    const tdp_status st = gn_check(plan, C, groups, 0, &p);
    if (st != TDP_OK) return st;
    if (!(eps >= 0.f) || (act != TDP_ACT_NONE && act != TDP_ACT_SILU))
        return tdp_fail(TDP_ERR_INVALID_ARG, "need eps >= 0 and a known act");
    if (plan->g.B == 0) return tdp_ok();
    if (!x || !y || !mean || !rstd || !ws || ws_bytes < p.bytes)
        return tdp_fail(TDP_ERR_INVALID_ARG, "null x, y, mean, rstd or ws, or ws too small");
    if (!tdp_aligned(x, 16) || !tdp_aligned(y, 16) || !tdp_aligned(gamma, 16) || !tdp_aligned(beta, 16) ||
        !tdp_aligned(mean, 4) || !tdp_aligned(rstd, 4) || !tdp_aligned(ws, 256))
        return tdp_fail(TDP_ERR_MISALIGNED, "x, y, gamma and beta need 16-byte, mean and rstd 4-byte, ws 256-byte alignment");
    gn_args a = {};
    a.C = C;
    a.G = groups;
    a.eps = eps;
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    const cudaError_t err = gn_dispatch<0>(plan->g, p, a, act, ws, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}

extern "C" tdp_status tdp_group_norm_grad(tdp_plan_t plan, int32_t C, int32_t groups, int32_t act, const void *x,
                                          const void *gamma, const void *beta, const float *mean, const float *rstd,
                                          const void *dy, void *dx, float *dgamma, float *dbeta, void *ws,
                                          int64_t ws_bytes, tdp_stream_t stream)
{
    gn_plan p;
    const tdp_status st = gn_check(plan, C, groups, 1, &p);
    if (st != TDP_OK) return st;
    if (act != TDP_ACT_NONE && act != TDP_ACT_SILU) return tdp_fail(TDP_ERR_INVALID_ARG, "unknown act");
    if ((dgamma == nullptr) != (dbeta == nullptr))
        return tdp_fail(TDP_ERR_INVALID_ARG, "dgamma and dbeta go together");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (plan->g.B == 0) {
        cudaError_t err = cudaSuccess;
        if (dgamma) err = cudaMemsetAsync(dgamma, 0, (size_t)C * 4, s);
        if (dbeta && err == cudaSuccess) err = cudaMemsetAsync(dbeta, 0, (size_t)C * 4, s);
        return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
    }
    if (!x || !dy || !dx || !mean || !rstd || !ws || ws_bytes < p.bytes)
        return tdp_fail(TDP_ERR_INVALID_ARG, "null x, dy, dx, mean, rstd or ws, or ws too small");
    if (!tdp_aligned(x, 16) || !tdp_aligned(dy, 16) || !tdp_aligned(dx, 16) || !tdp_aligned(gamma, 16) ||
        !tdp_aligned(beta, 16) || !tdp_aligned(mean, 4) || !tdp_aligned(rstd, 4) || !tdp_aligned(dgamma, 4) ||
        !tdp_aligned(dbeta, 4) || !tdp_aligned(ws, 256))
        return tdp_fail(TDP_ERR_MISALIGNED, "x, dy, dx, gamma and beta need 16-byte, fp32 buffers 4-byte, ws 256-byte alignment");
    gn_args a = {};
    a.C = C;
    a.G = groups;
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.dy = dy;
    a.y = dx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    const cudaError_t err = gn_dispatch<1>(plan->g, p, a, act, ws, s);
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}
