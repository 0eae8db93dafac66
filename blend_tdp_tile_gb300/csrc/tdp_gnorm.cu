// tdp_gnorm.cu -- group normalisation of every (tile, item), channels last, with an
// activation, and its gradients.
//
// Over the n = T_t * C/groups values of a group: mean, rstd = 1/sqrt(var + eps),
// z = (x - mean) * rstd * gamma + beta, y = act(z).  With h = (x - mean) * rstd,
// dz = dy * act'(z) and g = dz * gamma the gradient is
//   dx = rstd * (g - mean(g) - h * mean(g * h)),  dgamma = sum dz * h,  dbeta = sum dz.
//
// Three launches each way: per-channel sums of chunks of rows; their join; the elementwise
// pass.  The moments of a chunk are kept as (mean, sum of squared deviations) and joined by
// T. Chan's rule, so that a mean far from zero costs no digits; every join runs in a fixed
// order.
#include <algorithm>

#include "tdp.h"
#include "tdp_internal.h"
#include "tdp_rows.cuh"

namespace {

constexpr int kGnThreads = 256;
constexpr int kGnRows = 256;      // rows of a chunk

// ACT'(z) and ACT(z); SiLU is z * s, s = 1 / (1 + exp(-z)).
__device__ __forceinline__ float sigmoidf(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// exp(-z) past 2^126 makes the fast division return 0 / inf = 0 in the forward and s = 0 in the
// gradient: SiLU's limits.
template <int ACT>
__device__ __forceinline__ float act(float z) { return ACT ? z * sigmoidf(z) : z; }
template <int ACT>
__device__ __forceinline__ float act_grad(float z)
{
    if (!ACT) return 1.f;
    const float s = sigmoidf(z);
    return s * (1.f + z * (1.f - s));
}

struct gn_args {
    int32_t C, G, chunks;       // channels, groups, chunks per segment
    float eps;
    const void *x, *gamma, *beta, *dy;
    void *y;                    // y or dx
    float *mean, *rstd;         // [segments, G]
    float *dgamma, *dbeta;      // [C]
    float *part;                // [segments, chunks, C, 2]
    float *coef;                // [segments, C, 2] (gradient: sums over the segment)
};

// Column of 16-byte vectors and first row of this thread: vectors of a row side by side,
// then rows; blockIdx.y takes further vectors of rows wider than the block.
struct gn_lane {
    int32_t col, row, step;
    bool on;
};
__device__ __forceinline__ gn_lane gn_lane_of(int32_t CV)
{
    const int32_t w = CV < kGnThreads ? CV : kGnThreads;
    gn_lane l;
    l.step = kGnThreads / w;
    l.row = threadIdx.x / w;
    l.col = blockIdx.y * kGnThreads + threadIdx.x % w;
    l.on = l.row < l.step && l.col < CV;
    return l;
}

// Sums of a chunk's rows per channel.  Forward (GRAD = 0): mean and squared deviations,
// each thread about its own first value.  Gradient: sum dz, sum dz * h.
template <int BF16, int GRAD, int ACT>
__global__ void __launch_bounds__(kGnThreads)
tdp_gn_sums_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    using E = tdp_elem<BF16>;
    constexpr int V = E::kVec;
    __shared__ float red[kGnThreads * V * 2];
    const int32_t s = blockIdx.x / a.chunks, ch = blockIdx.x % a.chunks;
    const tdp_seg seg = tdp_seg_at(g, s);
    const int64_t r0 = (int64_t)ch * kGnRows;
    const int32_t rows = (int32_t)min((int64_t)kGnRows, seg.T - r0);
    const int32_t CV = a.C / V, cg = a.C / a.G;
    const gn_lane l = gn_lane_of(CV);
    tdp_pdl_trigger();
    tdp_pdl_wait();
    if (rows <= 0) return;
    float p[V], s1[V], s2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = s1[j] = s2[j] = 0.f;
    int32_t n = 0;
    if (l.on) {
        const uint4 *x = reinterpret_cast<const uint4 *>(a.x) + (seg.row0 + r0) * CV + l.col;
        if (!GRAD) {
            for (int32_t r = l.row; r < rows; r += l.step, ++n) {
                float f[V];
                E::unpack(x[(int64_t)r * CV], f);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (n == 0) p[j] = f[j];
                    const float d = f[j] - p[j];
                    s1[j] += d;
                    s2[j] += d * d;
                }
            }
            if (n > 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float m = s1[j] / n;
                    s2[j] -= s1[j] * m;         // squared deviations from the thread's mean
                    s1[j] = p[j] + m;
                }
            }
        } else {
            const uint4 *dy = reinterpret_cast<const uint4 *>(a.dy) + (seg.row0 + r0) * CV + l.col;
            float mu[V], rs[V], ga[V], be[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int32_t c = l.col * V + j;
                mu[j] = a.mean[(int64_t)s * a.G + c / cg];
                rs[j] = a.rstd[(int64_t)s * a.G + c / cg];
                ga[j] = a.gamma ? (float)reinterpret_cast<const typename E::type *>(a.gamma)[c] : 1.f;
                be[j] = a.beta ? (float)reinterpret_cast<const typename E::type *>(a.beta)[c] : 0.f;
            }
            for (int32_t r = l.row; r < rows; r += l.step) {
                float f[V], d[V];
                E::unpack(x[(int64_t)r * CV], f);
                E::unpack(dy[(int64_t)r * CV], d);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float h = (f[j] - mu[j]) * rs[j];
                    const float dz = d[j] * act_grad<ACT>(h * ga[j] + be[j]);
                    s1[j] += dz;
                    s2[j] += dz * h;
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        red[(threadIdx.x * V + j) * 2] = s1[j];
        red[(threadIdx.x * V + j) * 2 + 1] = s2[j];
    }
    __syncthreads();
    // the first row lane joins the lanes of its channels, in order
    if (l.on && l.row == 0) {
        const int32_t w = CV < kGnThreads ? CV : kGnThreads;
        float *out = a.part + (((int64_t)s * a.chunks + ch) * a.C + l.col * V) * 2;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float A = s1[j], Q = s2[j], N = (float)((rows + l.step - 1) / l.step);
            for (int32_t k = 1; k < l.step && k < rows; ++k) {
                const float *o = red + ((threadIdx.x + k * w) * V + j) * 2;
                if (GRAD) {
                    A += o[0];
                    Q += o[1];
                } else {
                    const float m = (float)((rows - k + l.step - 1) / l.step), d = o[0] - A;
                    A += d * (m / (N + m));
                    Q += o[1] + d * d * (N * m / (N + m));
                    N += m;
                }
            }
            out[2 * j] = A;
            out[2 * j + 1] = Q;
        }
    }
}

// One warp per (segment, group): the group's moments from its channels' and chunks' (mean, squared
// deviations): first the mean, then the deviations about it.
__global__ void __launch_bounds__(kGnThreads)
tdp_gn_moments_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const int64_t w = ((int64_t)blockIdx.x * kGnThreads + threadIdx.x) >> 5;
    const int32_t lane = threadIdx.x & 31;
    if (w >= (int64_t)g.nt * g.B * a.G) return;
    const int32_t s = (int32_t)(w / a.G), gr = (int32_t)(w % a.G);
    const tdp_seg seg = tdp_seg_at(g, s);
    const int32_t cg = a.C / a.G, chunks = (int32_t)((seg.T + kGnRows - 1) / kGnRows);
    const float *part = a.part + ((int64_t)s * a.chunks * a.C + gr * cg) * 2;
    const float n = (float)seg.T * cg;
    float mean = 0.f;
    for (int32_t i = lane; i < chunks * cg; i += 32) {
        const int32_t k = i / cg;
        const float m = (float)min((int64_t)kGnRows, seg.T - (int64_t)k * kGnRows);
        mean += part[((int64_t)k * a.C + i % cg) * 2] * (m / n);
    }
    for (int o = 16; o; o >>= 1) mean += __shfl_xor_sync(~0u, mean, o);
    float q = 0.f;
    for (int32_t i = lane; i < chunks * cg; i += 32) {
        const int32_t k = i / cg;
        const float m = (float)min((int64_t)kGnRows, seg.T - (int64_t)k * kGnRows);
        const float *o = part + ((int64_t)k * a.C + i % cg) * 2;
        q += o[1] + m * (o[0] - mean) * (o[0] - mean);
    }
    for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(~0u, q, o);
    if (lane == 0) {
        a.mean[w] = mean;
        a.rstd[w] = 1.f / sqrtf(q / n + a.eps);
    }
}

// One thread per (segment, channel): the chunks' gradient sums of the segment.
__global__ void __launch_bounds__(kGnThreads)
tdp_gn_join_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kGnThreads + threadIdx.x;
    if (i >= (int64_t)g.nt * g.B * a.C) return;
    const int32_t s = (int32_t)(i / a.C), c = (int32_t)(i % a.C);
    const int32_t chunks = (int32_t)((tdp_seg_at(g, s).T + kGnRows - 1) / kGnRows);
    float s1 = 0.f, s2 = 0.f;
    for (int32_t k = 0; k < chunks; ++k) {
        const float *o = a.part + (((int64_t)s * a.chunks + k) * a.C + c) * 2;
        s1 += o[0];
        s2 += o[1];
    }
    a.coef[2 * i] = s1;
    a.coef[2 * i + 1] = s2;
}

// One warp per channel: dgamma and dbeta, the segments' sums joined.
__global__ void __launch_bounds__(kGnThreads)
tdp_gn_param_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const int32_t c = (int32_t)(((int64_t)blockIdx.x * kGnThreads + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    if (c >= a.C) return;
    float s1 = 0.f, s2 = 0.f;
    for (int32_t s = lane; s < g.nt * g.B; s += 32) {
        s1 += a.coef[((int64_t)s * a.C + c) * 2];
        s2 += a.coef[((int64_t)s * a.C + c) * 2 + 1];
    }
    for (int o = 16; o; o >>= 1) {
        s1 += __shfl_xor_sync(~0u, s1, o);
        s2 += __shfl_xor_sync(~0u, s2, o);
    }
    if (lane == 0) {
        a.dbeta[c] = s1;
        a.dgamma[c] = s2;
    }
}

// The elementwise pass: y from x, or dx from x and dy.
template <int BF16, int GRAD, int ACT>
__global__ void __launch_bounds__(kGnThreads)
tdp_gn_apply_kernel(const __grid_constant__ tdp_geom g, const gn_args a)
{
    using E = tdp_elem<BF16>;
    constexpr int V = E::kVec;
    const int32_t s = blockIdx.x / a.chunks, ch = blockIdx.x % a.chunks;
    const tdp_seg seg = tdp_seg_at(g, s);
    const int64_t r0 = (int64_t)ch * kGnRows;
    const int32_t rows = (int32_t)min((int64_t)kGnRows, seg.T - r0);
    const int32_t CV = a.C / V, cg = a.C / a.G;
    const gn_lane l = gn_lane_of(CV);
    tdp_pdl_trigger();
    tdp_pdl_wait();
    if (rows <= 0 || !l.on) return;
    float mu[V], rs[V], ga[V], be[V], m1[V], m2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int32_t c = l.col * V + j, gr = c / cg;
        mu[j] = a.mean[(int64_t)s * a.G + gr];
        rs[j] = a.rstd[(int64_t)s * a.G + gr];
        ga[j] = a.gamma ? (float)reinterpret_cast<const typename E::type *>(a.gamma)[c] : 1.f;
        be[j] = a.beta ? (float)reinterpret_cast<const typename E::type *>(a.beta)[c] : 0.f;
        m1[j] = m2[j] = 0.f;
        if (GRAD) {     // means of g and g * h over the group
            if (j > 0 && gr == (c - 1) / cg) {
                m1[j] = m1[j - 1];
                m2[j] = m2[j - 1];
            } else {
                for (int32_t k = gr * cg; k < (gr + 1) * cg; ++k) {
                    const float w = a.gamma ? (float)reinterpret_cast<const typename E::type *>(a.gamma)[k] : 1.f;
                    m1[j] += w * a.coef[((int64_t)s * a.C + k) * 2];
                    m2[j] += w * a.coef[((int64_t)s * a.C + k) * 2 + 1];
                }
                m1[j] /= (float)seg.T * cg;
                m2[j] /= (float)seg.T * cg;
            }
        }
    }
    const int64_t at = (seg.row0 + r0) * CV + l.col;
    const uint4 *x = reinterpret_cast<const uint4 *>(a.x) + at;
    const uint4 *dy = reinterpret_cast<const uint4 *>(a.dy) + at;
    uint4 *y = reinterpret_cast<uint4 *>(a.y) + at;
    for (int32_t r = l.row; r < rows; r += l.step) {
        float f[V], d[V];
        E::unpack(x[(int64_t)r * CV], f);
        if (GRAD) E::unpack(dy[(int64_t)r * CV], d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float h = (f[j] - mu[j]) * rs[j], z = h * ga[j] + be[j];
            f[j] = GRAD ? rs[j] * (d[j] * act_grad<ACT>(z) * ga[j] - m1[j] - h * m2[j]) : act<ACT>(z);
        }
        y[(int64_t)r * CV] = E::pack(f);
    }
}

int64_t gn_part_bytes(const tdp_geom &g, int32_t C, int64_t chunks)
{
    return (int64_t)g.nt * g.B * chunks * C * 8;
}

// Workspace: part, then coef.
tdp_status gn_check(tdp_plan_t plan, int32_t C, int32_t groups, int64_t *bytes, int64_t *chunks)
{
    if (!plan) return tdp_fail(TDP_ERR_INVALID_ARG, "null plan");
    const tdp_geom &g = plan->g;
    if (C < 1 || groups < 1 || C % groups != 0)
        return tdp_fail(TDP_ERR_INVALID_ARG, "need groups >= 1 dividing C");
    if (((int64_t)C * g.esize) % 16 != 0)
        return tdp_fail(TDP_ERR_MISALIGNED, "C * element size must be a multiple of 16 bytes");
    *chunks = (tdp_max_tile_tokens(g) + kGnRows - 1) / kGnRows;
    if ((int64_t)g.nt * g.B * *chunks > 0x7fffffffLL || (int64_t)C * g.esize / 16 > (int64_t)kGnThreads * 65535 ||
        (int64_t)g.B * g.total > ((int64_t)1 << 56) / C)
        return tdp_fail(TDP_ERR_TOO_LARGE, "group normalisation beyond index ranges");
    *bytes = gn_part_bytes(g, C, *chunks) + (int64_t)g.nt * g.B * C * 8;
    return TDP_OK;
}

template <int GRAD>
cudaError_t gn_launch(const tdp_geom &g, gn_args a, int32_t act, cudaStream_t s)
{
    const int V = g.dtype == TDP_BF16 ? 8 : 4;
    const int32_t segs = g.nt * g.B;
    const dim3 grid((unsigned)(segs * a.chunks), (unsigned)((a.C / V + kGnThreads - 1) / kGnThreads));
    auto launch = [&](auto *k, dim3 gr) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = gr;
        cfg.blockDim = dim3(kGnThreads);
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, k, g, a);
    };
    auto blocks = [&](int64_t threads) { return dim3((unsigned)((threads + kGnThreads - 1) / kGnThreads)); };
    cudaError_t err = g.dtype == TDP_BF16
                          ? launch(act ? tdp_gn_sums_kernel<1, GRAD, 1> : tdp_gn_sums_kernel<1, GRAD, 0>, grid)
                          : launch(act ? tdp_gn_sums_kernel<0, GRAD, 1> : tdp_gn_sums_kernel<0, GRAD, 0>, grid);
    if (err == cudaSuccess)
        err = GRAD ? launch(tdp_gn_join_kernel, blocks((int64_t)segs * a.C))
                   : launch(tdp_gn_moments_kernel, blocks((int64_t)segs * a.G * 32));
    if (err == cudaSuccess && GRAD && a.dgamma) err = launch(tdp_gn_param_kernel, blocks((int64_t)a.C * 32));
    if (err == cudaSuccess)
        err = g.dtype == TDP_BF16
                  ? launch(act ? tdp_gn_apply_kernel<1, GRAD, 1> : tdp_gn_apply_kernel<1, GRAD, 0>, grid)
                  : launch(act ? tdp_gn_apply_kernel<0, GRAD, 1> : tdp_gn_apply_kernel<0, GRAD, 0>, grid);
    return err;
}

}  // namespace

extern "C" tdp_status tdp_group_norm_workspace(tdp_plan_t plan, int32_t C, int32_t groups, int64_t *bytes)
{
    int64_t chunks, need;
    if (!bytes) return tdp_fail(TDP_ERR_INVALID_ARG, "null bytes");
    const tdp_status st = gn_check(plan, C, groups, &need, &chunks);
    if (st != TDP_OK) return st;
    *bytes = need;
    return tdp_ok();
}

extern "C" tdp_status tdp_group_norm(tdp_plan_t plan, int32_t C, int32_t groups, float eps, int32_t act, const void *x,
                                     const void *gamma, const void *beta, void *y, float *mean, float *rstd, void *ws,
                                     int64_t ws_bytes, tdp_stream_t stream)
{
    int64_t chunks, need;
    const tdp_status st = gn_check(plan, C, groups, &need, &chunks);
    if (st != TDP_OK) return st;
    if (!(eps >= 0.f) || (act != TDP_ACT_NONE && act != TDP_ACT_SILU))
        return tdp_fail(TDP_ERR_INVALID_ARG, "need eps >= 0 and a known act");
    if (plan->g.B == 0) return tdp_ok();
    if (!x || !y || !mean || !rstd || !ws || ws_bytes < need)
        return tdp_fail(TDP_ERR_INVALID_ARG, "null x, y, mean, rstd or ws, or ws too small");
    if (!tdp_aligned(x, 16) || !tdp_aligned(y, 16) || !tdp_aligned(gamma, 16) || !tdp_aligned(beta, 16) ||
        !tdp_aligned(mean, 4) || !tdp_aligned(rstd, 4) || !tdp_aligned(ws, 256))
        return tdp_fail(TDP_ERR_MISALIGNED, "x, y, gamma and beta need 16-byte, mean and rstd 4-byte, ws 256-byte alignment");
    gn_args a = {};
    a.C = C;
    a.G = groups;
    a.chunks = (int32_t)chunks;
    a.eps = eps;
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.part = reinterpret_cast<float *>(ws);
    const cudaError_t err = gn_launch<0>(plan->g, a, act, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}

extern "C" tdp_status tdp_group_norm_grad(tdp_plan_t plan, int32_t C, int32_t groups, int32_t act, const void *x,
                                          const void *gamma, const void *beta, const float *mean, const float *rstd,
                                          const void *dy, void *dx, float *dgamma, float *dbeta, void *ws,
                                          int64_t ws_bytes, tdp_stream_t stream)
{
    int64_t chunks, need;
    const tdp_status st = gn_check(plan, C, groups, &need, &chunks);
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
    if (!x || !dy || !dx || !mean || !rstd || !ws || ws_bytes < need)
        return tdp_fail(TDP_ERR_INVALID_ARG, "null x, dy, dx, mean, rstd or ws, or ws too small");
    if (!tdp_aligned(x, 16) || !tdp_aligned(dy, 16) || !tdp_aligned(dx, 16) || !tdp_aligned(gamma, 16) ||
        !tdp_aligned(beta, 16) || !tdp_aligned(mean, 4) || !tdp_aligned(rstd, 4) || !tdp_aligned(dgamma, 4) ||
        !tdp_aligned(dbeta, 4) || !tdp_aligned(ws, 256))
        return tdp_fail(TDP_ERR_MISALIGNED, "x, dy, dx, gamma and beta need 16-byte, fp32 buffers 4-byte, ws 256-byte alignment");
    gn_args a = {};
    a.C = C;
    a.G = groups;
    a.chunks = (int32_t)chunks;
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.dy = dy;
    a.y = dx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.part = reinterpret_cast<float *>(ws);
    a.coef = a.part + gn_part_bytes(plan->g, C, chunks) / 4;
    const cudaError_t err = gn_launch<1>(plan->g, a, act, s);
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}
