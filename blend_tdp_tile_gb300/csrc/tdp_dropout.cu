// tdp_dropout.cu -- residual + dropout from a counter-based generator, and its gradient.
//
// out_i = res_i + (w_i >= thr ? x_i / (1 - p) : 0), thr = round(p * 2^32), w_i = word i % 4 of
// Philox4x32-10 of counter {i/4, offset} and key seed (J. Salmon, M. Moraes, R. Dror,
// D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011): the mask is a function
// of the element's index, so the gradient computes it again and nothing is stored.
#include <algorithm>
#include <cmath>

#include "tdp.h"
#include "tdp_internal.h"
#include "tdp_rows.cuh"

namespace {

constexpr int kDropThreads = 256;
constexpr uint32_t kPhilox0 = 0xD2511F53u, kPhilox1 = 0xCD9E8D57u;

// Round keys of Philox4x32-10: the key and its nine bumps.
struct philox_keys {
    uint32_t k0[10], k1[10];
    __device__ __forceinline__ explicit philox_keys(uint64_t seed)
    {
#pragma unroll
        for (int r = 0; r < 10; ++r) {
            k0[r] = (uint32_t)seed + r * 0x9E3779B9u;
            k1[r] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
        }
    }
};

// What the first two rounds of a counter {index, offset} owe to the offset and the index's high word alone: two of the
// twenty products, the same for four billion counters.
struct philox_head {
    uint32_t hi, c1, c0x;           // index's high word; round 1's input c1; hi(q0) ^ k1 of round 1
    uint32_t lo;                    // lo(q0)
    __device__ __forceinline__ void at(uint32_t high, uint64_t offset, const philox_keys &k)
    {
        const uint64_t p1 = (uint64_t)(uint32_t)offset * kPhilox1, q0 = (uint64_t)((uint32_t)(p1 >> 32) ^ high ^ k.k0[0]) * kPhilox0;
        hi = high;
        c1 = (uint32_t)p1;
        c0x = (uint32_t)(q0 >> 32) ^ k.k1[1];
        lo = (uint32_t)q0;
    }
};

// Ten rounds of two 32x32 -> 64-bit products.
__device__ __forceinline__ uint4 philox10(uint32_t index, uint64_t offset, const philox_head &h, const philox_keys &k)
{
    const uint64_t f0 = (uint64_t)index * kPhilox0, f1 = (uint64_t)((uint32_t)(f0 >> 32) ^ (uint32_t)(offset >> 32) ^ k.k1[0]) * kPhilox1;
    uint32_t c0 = (uint32_t)(f1 >> 32) ^ h.c1 ^ k.k0[1], c1 = (uint32_t)f1, c2 = h.c0x ^ (uint32_t)f0, c3 = h.lo;
#pragma unroll
    for (int r = 2; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)c0 * kPhilox0, p1 = (uint64_t)c2 * kPhilox1;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k.k0[r];
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k.k1[r];
        c3 = (uint32_t)p0;
    }
    return make_uint4(c0, c1, c2, c3);
}

// The words of vector i's elements.
template <int V>
__device__ __forceinline__ void drop_words(int64_t i, uint64_t offset, philox_head &h, const philox_keys &k, uint32_t *w)
{
    const uint64_t first = (uint64_t)i * (V / 4);           // of one or two counters, an even one where two: one high word
    if ((uint32_t)(first >> 32) != h.hi) h.at((uint32_t)(first >> 32), offset, k);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
        const uint4 u = philox10((uint32_t)first + j, offset, h, k);
        w[4 * j] = u.x;
        w[4 * j + 1] = u.y;
        w[4 * j + 2] = u.z;
        w[4 * j + 3] = u.w;
    }
}

// 16-byte vectors (4 fp32 or 8 bf16 elements: one or two counters); the vector that
// holds the end is done element by element by one thread.  `thr` is at most 2^32 - 1; p = 1 has all = 1.
// 105 million bf16 elements: 102 us, 6.2 TB/s, near the memory's rate, with one vector of each input ahead of the
// generator (107 with two); without the residual (the gradient) three: 92 us, 4.6 TB/s, for 97 with one.  There the
// generator's wide products, 18 of 20 a thread's own, keep the integer multiplier busy.
template <int BF16, int RES>
__global__ void __launch_bounds__(kDropThreads)
tdp_dropout_kernel(int64_t n, uint32_t thr, int all, float scale, const uint64_t *__restrict__ rng, const void *x,
                   const void *res, void *out)
{
    using E = tdp_elem<BF16>;
    constexpr int V = E::kVec, U = RES ? 1 : 3;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const uint64_t offset = rng[1];
    const philox_keys keys(rng[0]);
    philox_head head;
    head.at(0, offset, keys);
    const int64_t nv = n / V;
    const uint4 *xv = reinterpret_cast<const uint4 *>(x), *rv = reinterpret_cast<const uint4 *>(res);
    for (int64_t i0 = (int64_t)blockIdx.x * (kDropThreads * U) + threadIdx.x; i0 < nv; i0 += (int64_t)gridDim.x * (kDropThreads * U)) {
        uint4 a[U], r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kDropThreads;
            if (i < nv) {
                a[u] = __ldcs(xv + i);
                if (RES) r[u] = __ldcs(rv + i);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kDropThreads;
            if (i >= nv) break;
            uint32_t w[V];
            float f[V], g[V];
            drop_words<V>(i, offset, head, keys, w);
            E::unpack(a[u], f);
            if (RES) E::unpack(r[u], g);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float k = w[j] >= thr && !all ? f[j] * scale : 0.f;
                f[j] = RES ? g[j] + k : k;
            }
            __stcs(reinterpret_cast<uint4 *>(out) + i, E::pack(f));
        }
    }
    if (n % V != 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        using T = typename E::type;
        uint32_t w[V];
        drop_words<V>(nv, offset, head, keys, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t e = nv * V + j;
            if (e >= n) break;
            const float k = w[j] >= thr && !all ? (float)reinterpret_cast<const T *>(x)[e] * scale : 0.f;
            reinterpret_cast<T *>(out)[e] = (T)(RES ? (float)reinterpret_cast<const T *>(res)[e] + k : k);
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
    const int all = thr > 0xffffffffull;
    const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    const int64_t step = (int64_t)kDropThreads * (plan->g.dtype == TDP_BF16 ? 8 : 4);
    const unsigned grid = (unsigned)std::min<int64_t>((n + step - 1) / step, 152 * 64);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto *kernel = plan->g.dtype == TDP_BF16 ? (res ? tdp_dropout_kernel<1, 1> : tdp_dropout_kernel<1, 0>)
                                             : (res ? tdp_dropout_kernel<0, 1> : tdp_dropout_kernel<0, 0>);
    const cudaError_t err = tdp_launch(true, kernel, grid, kDropThreads, s, n, (uint32_t)thr, all, scale, rng, x, res, out);
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
