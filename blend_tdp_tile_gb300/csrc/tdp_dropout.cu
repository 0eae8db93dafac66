// tdp_dropout.cu -- residual + dropout from a counter-based generator, and its gradient.
//
// out_i = res_i + (w_i >= thr ? x_i / (1 - p) : 0), thr = round(p * 2^32), w_i = word i % 4 of
// Philox4x32-10 of counter {i/4, offset} and key seed (J. Salmon, M. Moraes, R. Dror,
// D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011): the mask is a function
// of the element's index, so the gradient computes it again and nothing is stored.
#include <cmath>

#include "tdp.h"
#include "tdp_internal.h"
#include "tdp_rows.cuh"

namespace {

constexpr int kDropThreads = 256;

// Philox4x32-10: ten rounds of two 32x32 -> 64-bit products, the key bumped between rounds.
__device__ __forceinline__ uint4 philox10(uint64_t index, uint64_t offset, uint64_t seed)
{
    uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// One 16-byte vector a thread and step (4 fp32 or 8 bf16 elements: one or two counters); the
// vector that holds the end is done element by element.
template <int BF16, int RES>
__global__ void __launch_bounds__(kDropThreads)
tdp_dropout_kernel(int64_t n, uint64_t thr, float scale, const uint64_t *__restrict__ rng, const void *x,
                   const void *res, void *out)
{
    using E = tdp_elem<BF16>;
    constexpr int V = E::kVec;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const uint64_t seed = rng[0], offset = rng[1];
    const int64_t nv = (n + V - 1) / V;
    for (int64_t i = (int64_t)blockIdx.x * kDropThreads + threadIdx.x; i < nv; i += (int64_t)gridDim.x * kDropThreads) {
        uint32_t w[V];
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const uint4 u = philox10((uint64_t)i * (V / 4) + j, offset, seed);
            w[4 * j] = u.x;
            w[4 * j + 1] = u.y;
            w[4 * j + 2] = u.z;
            w[4 * j + 3] = u.w;
        }
        if ((i + 1) * V <= n) {
            float f[V], r[V];
            E::unpack(reinterpret_cast<const uint4 *>(x)[i], f);
            if (RES) E::unpack(reinterpret_cast<const uint4 *>(res)[i], r);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float k = w[j] >= thr ? f[j] * scale : 0.f;
                f[j] = RES ? r[j] + k : k;
            }
            reinterpret_cast<uint4 *>(out)[i] = E::pack(f);
        } else {
            for (int64_t e = i * V; e < n; ++e) {
                using T = typename E::type;
                const float k = w[e - i * V] >= thr ? (float)reinterpret_cast<const T *>(x)[e] * scale : 0.f;
                reinterpret_cast<T *>(out)[e] = (T)(RES ? (float)reinterpret_cast<const T *>(res)[e] + k : k);
            }
        }
    }
}

tdp_status dropout(tdp_plan_t plan, int64_t n, double p, const uint64_t *rng, const void *x, const void *res, void *out,
                   tdp_stream_t stream)
{
    if (!plan) return tdp_fail(TDP_ERR_INVALID_ARG, "null plan");
    if (n < 0 || !(p >= 0.0 && p <= 1.0)) return tdp_fail(TDP_ERR_INVALID_ARG, "need n >= 0 and 0 <= p <= 1");
    if (n == 0) return tdp_ok();
    if (!rng || !x || !out) return tdp_fail(TDP_ERR_INVALID_ARG, "null rng, input or output");
    if (!tdp_aligned(rng, 8) || !tdp_aligned(x, 16) || !tdp_aligned(out, 16) || !tdp_aligned(res, 16))
        return tdp_fail(TDP_ERR_MISALIGNED, "elements need 16-byte, rng 8-byte alignment");
    if (n > ((int64_t)1 << 56)) return tdp_fail(TDP_ERR_TOO_LARGE, "n above 2^56");
    const uint64_t thr = (uint64_t)std::llrint(p * 4294967296.0);
    const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    const int V = plan->g.dtype == TDP_BF16 ? 8 : 4;
    const int64_t blocks = ((n + V - 1) / V + kDropThreads - 1) / kDropThreads;
    const unsigned grid = (unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto *kernel = plan->g.dtype == TDP_BF16 ? (res ? tdp_dropout_kernel<1, 1> : tdp_dropout_kernel<1, 0>)
                                             : (res ? tdp_dropout_kernel<0, 1> : tdp_dropout_kernel<0, 0>);
    const cudaError_t err = tdp_launch(true, kernel, grid, kDropThreads, s, n, thr, scale, rng, x, res, out);
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}

}  // namespace

extern "C" tdp_status tdp_dropout_add(tdp_plan_t plan, int64_t n, double p, const uint64_t *rng, const void *x,
                                      const void *res, void *out, tdp_stream_t stream)
{
    return dropout(plan, n, p, rng, x, res, out, stream);
}

extern "C" tdp_status tdp_dropout_grad(tdp_plan_t plan, int64_t n, double p, const uint64_t *rng, const void *dout,
                                       void *dx, tdp_stream_t stream)
{
    return dropout(plan, n, p, rng, dout, nullptr, dx, stream);
}
