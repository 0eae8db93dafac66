// tdp_matmul8.cu -- product of 8-bit rows and 8-bit weights (e4m3), a scale a row and a channel, bias and residual.
//
// out[r, n] = xs_r ws_n sum_k x8[r, k] w8[n, k] + bias_n + res[r, n].  Products of e4m3 values are exact in fp32, sums are
// fp32 on the tensor cores (tcgen05, kind f8f6f4); scales, bias and residual come in fp32 behind the sum, one rounding
// at the end.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "tdp.h"
#include "tdp_host.h"
#include "tdp_internal.h"
#include "tdp_matmul8.cuh"
#include "tdp_tensor_map.h"

namespace tdp_m8 {

// Tiles of 128 channels by NT rows, one a block, K split over the blocks of a cluster.
//
// Channels are the lanes and rows the columns of the accumulator, so that few rows make a small tile: the weights' bytes bound
// such a product, and a cluster's blocks each bring a part of K.  Warps 0-3 take the sums out of tensor memory, warp 4 loads, warp 5
// issues the products.  The parts are joined through distributed shared memory, each block adding up its share of the
// rows in the order of the parts.
template <int NT>
struct tile_smem {
    static constexpr int kStage = 16384 + NT * 128;
    static constexpr int kStages = NT <= 16 ? 5 : 4;        // two blocks an SM
    static constexpr int kBytes = 1024 + kStages * kStage;
    static_assert(kStages * kStage >= NT * 512, "the parts lie where the stages were");
};
constexpr int kTileThreads = 192;

template <int BF16, int NT>
__global__ void __launch_bounds__(kTileThreads)
tdp_matmul8_tile_kernel(const __grid_constant__ args a, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x)
{
    using SM = tile_smem<NT>;
    constexpr int NST = SM::kStages;
    constexpr uint32_t kCols = NT < 32 ? 32 : NT;
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t bar_mem[2 * NST + 1];
    __shared__ float xs[NT];
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_flag, far_flag;
    volatile int *dead = &dead_flag;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u, full = smem_u32(bar_mem), empty = full + 8 * NST, done = empty + 8 * NST;
    const int32_t warp = warp_id(), lane = threadIdx.x & 31;
    if (warp == 5) tmem_alloc(smem_u32(&tmem_slot), kCols);
    if (threadIdx.x == 0) {
        dead_flag = far_flag = 0;
        for (int i = 0; i < 2 * NST + 1; ++i) mbar_init(full + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = tmem_slot;
    tdp_pdl_trigger();
    tdp_pdl_wait();

    const uint32_t split = cluster_size(), rank = cluster_rank();
    const int32_t tile = blockIdx.x / split, tc = tile % a.tiles_c;
    const int32_t ch0 = tc * 128;
    const int64_t row0 = (int64_t)(tile / a.tiles_c) * NT;
    const int32_t k0 = (int32_t)((int64_t)a.kb * rank / split), n = (int32_t)((int64_t)a.kb * (rank + 1) / split) - k0;
    using E = tdp_elem<BF16>;
    using T = typename E::type;
    const int32_t ch = ch0 + 2 * (threadIdx.x & 63);            // two channels of the output
    const bool in = ch < a.N;
    const T *bias = static_cast<const T *>(a.bias);
    float2 w = make_float2(0.f, 0.f), b = w;
    bool ok = true;
    int32_t made = 0;
    if (warp == 4) {
#pragma unroll 1
        for (; made < n; ++made) {
            const int32_t st = made % NST;
            if (!(ok = mbar_wait(empty + 8 * st, ((made / NST) & 1) ^ 1, dead))) break;
            if (elect_one()) {
                const uint32_t to = base + st * SM::kStage;
                mbar_expect(full + 8 * st, (uint32_t)(a.w_box + a.x_box) * kK);
                tma_load2(to, &map_w, full + 8 * st, (k0 + made) * kK, ch0);
                tma_load2(to + 16384, &map_x, full + 8 * st, (k0 + made) * kK, (int32_t)row0);
            }
            __syncwarp();
        }
        for (int32_t i = max(0, made - NST); i < made; ++i) landed(full + 8 * (i % NST), (i / NST) & 1);
    } else if (warp == 5) {
        constexpr uint32_t id = idesc8(128, NT);
#pragma unroll 1
        for (int32_t i = 0; i < n; ++i) {
            const int32_t st = i % NST;
            if (!(ok = mbar_wait(full + 8 * st, (i / NST) & 1, dead))) break;
            fence_after();
            if (elect_one()) {
                const uint32_t w = desc_rows(base + st * SM::kStage), x = desc_rows(base + st * SM::kStage + 16384);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma8(tm, w + 2 * k, x + 2 * k, id, i > 0 || k > 0);
                mma_commit(empty + 8 * st);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(done);
        __syncwarp();
        landed(done, 0);
    } else {
        // what the end takes besides the sums, asked for under the products
        if (threadIdx.x < NT) {
            const float x = row0 + threadIdx.x < a.rows ? __ldcg(a.xs + row0 + threadIdx.x) : 1.f;
            xs[threadIdx.x] = x;
            if (!plain_scale(x)) far_flag = 1;
        }
        if (in) {
            w = __ldcg(reinterpret_cast<const float2 *>(a.ws + ch));
            if (bias) b = make_float2((float)bias[ch], (float)bias[ch + 1]);
        }
        ok = mbar_wait(done, 0, dead);
        fence_after();
    }
    __syncwarp();
    // No block reads its stages any more, nothing is on its way to them: the parts take their place.
    if (split > 1) cluster_sync();
    else __syncthreads();
    // part[from][row of the block's share][channel]
    const int32_t share = NT / split, shift = __ffs(share) - 1;
    if (warp < 4) {
        ok = __all_sync(~0u, ok && !*dead);
        const uint32_t from = tm + ((uint32_t)warp << 21);
        constexpr int B = NT < 32 ? 16 : 32;
#pragma unroll 1
        for (int c0 = 0; c0 < NT; c0 += B) {
            uint32_t v[B];
            if (B == 16) tmem_ld16(from + c0, v);
            else tmem_ld32(from + c0, v);
            tmem_wait_ld();
            if (B == 16) tmem_have16(v);
            else tmem_have32(v);
#pragma unroll
            for (int c = 0; c < B; ++c) {
                if (!ok) v[c] = 0x7fffffffu;
                const uint32_t to = (c0 + c) >> shift, r = (c0 + c) & (share - 1);
                asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(at_rank(base + ((rank * share + r) * 128 + threadIdx.x) * 4, to)), "r"(v[c]) : "memory");
            }
        }
        fence_before();
    }
    __syncwarp();
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (warp < 4 && in) {
        constexpr int U = 4;                // rows whose residuals a thread has under way
        const float *part = reinterpret_cast<const float *>(raw + (base - smem_u32(raw))) + 2 * (threadIdx.x & 63);
        const int64_t first = row0 + (int64_t)rank * share;
        const int32_t end = (int32_t)min((int64_t)share, a.rows - first);
        auto rows_out = [&](auto any_far) {
            constexpr bool FAR = decltype(any_far)::value;
#pragma unroll 1
            for (int32_t r0 = threadIdx.x >> 6; r0 < end; r0 += 2 * U) {
                uint2 s[U];
                if (a.res) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const T *at = static_cast<const T *>(a.res) + (first + min(r0 + 2 * u, end - 1)) * a.N + ch;
                        if (BF16) s[u].x = *reinterpret_cast<const uint32_t *>(at);
                        else s[u] = *reinterpret_cast<const uint2 *>(at);
                    }
                }
                float2 sum[U];
#pragma unroll
                for (int u = 0; u < U; ++u) sum[u] = make_float2(0.f, 0.f);
                for (uint32_t f = 0; f < split; ++f) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float2 p = *reinterpret_cast<const float2 *>(part + ((f << shift) + min(r0 + 2 * u, end - 1)) * 128);
                        sum[u].x += p.x;
                        sum[u].y += p.y;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t r = r0 + 2 * u;
                    if (r >= end) break;
                    float2 v = sum[u];
                    const float x = xs[rank * share + r];
                    if (!FAR || plain_scale(x)) {
                        v.x = fmaf(v.x * x, w.x, b.x);
                        v.y = fmaf(v.y * x, w.y, b.y);
                    } else {
                        v.x = far_scaled(v.x, x, w.x, b.x);
                        v.y = far_scaled(v.y, x, w.y, b.y);
                    }
                    if (a.res) {
                        v.x += BF16 ? tdp_bf16_lo(s[u].x) : __uint_as_float(s[u].x);
                        v.y += BF16 ? tdp_bf16_hi(s[u].x) : __uint_as_float(s[u].y);
                    }
                    T *to = static_cast<T *>(a.out) + (first + r) * a.N + ch;
                    if (BF16) *reinterpret_cast<uint32_t *>(to) = tdp_pack_bf16x2(v.x, v.y);
                    else *reinterpret_cast<float2 *>(to) = v;
                }
            }
        };
        if (far_flag) rows_out(std::true_type{});
        else rows_out(std::false_type{});
    }
    fence_before();
    __syncthreads();
    if (warp == 5) tmem_free(tm, kCols);
}

// Tiles of 256 rows by 256 channels, each by a pair of blocks (cta_group::2), in turn.
//
// Each block brings 128 rows and 128 channels of a stage, and holds the sums of its rows against all 256 channels: half the
// shared-memory and L2 traffic of tiles that one block holds alone.  Warp 0 loads, warp 1 of the pair's first block issues the
// products of both, four warpgroups behind them take the sums out of one accumulator, a row and 64 channels a thread, while
// the next tile's are made in the other.
struct pair_smem {
    static constexpr int kStage = 32768;
    static constexpr int kStages = 5;
    static constexpr int kOut = 4096;           // two panels of a warp's outputs on their way to memory: 32 rows of 64 bytes
    static constexpr int kScales = 2048;        // a tile's scales and bias of 256 channels
    static constexpr int kBars = 8 * (2 * kStages + 5 + 32) + 8;
    // all that a block may have; the start is a multiple of 1024, as nothing but this lies in shared memory
    static constexpr int kBytes = 232448;
    static_assert(kStages * kStage + 16 * kOut + kScales + kBars <= kBytes - 512, "room for the stages");
};
constexpr int kPairThreads = 640;

template <int BF16, int RES>
__global__ void __launch_bounds__(kPairThreads, 1)
tdp_matmul8_pair_kernel(const __grid_constant__ args a, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ CUtensorMap map_o, const __grid_constant__ CUtensorMap map_r)
{
    using SM = pair_smem;
    using E = tdp_elem<BF16>;
    using T = typename E::type;
    constexpr int NST = SM::kStages;
    extern __shared__ __align__(1024) unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u, out_s = base + NST * SM::kStage;
    unsigned char *tail = raw + (base - smem_u32(raw)) + NST * SM::kStage + 16 * SM::kOut;
    float *scales = reinterpret_cast<float *>(tail);            // channels' scales, then their bias
    volatile int *dead = reinterpret_cast<int *>(tail + SM::kScales);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tail + SM::kScales + 4);
    const uint32_t full = smem_u32(tail + SM::kScales + 8), empty = full + 8 * NST, sums = empty + 8 * NST, taken = sums + 16, drain = taken + 16, added = drain + 8;
    const int32_t warp = warp_id(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (warp == 2) pair_alloc(smem_u32(tmem_slot), 512);
    if (threadIdx.x == 0) {
        *dead = 0;
        for (int i = 0; i < 2 * NST; ++i) mbar_init(full + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(sums + 8 * i, 1);
            mbar_init(taken + 8 * i, 32);       // sixteen warps of either block
        }
        mbar_init(drain, 1);
        for (int i = 0; i < 32; ++i) mbar_init(added + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    const uint32_t tm = *tmem_slot;
    tdp_pdl_trigger();
    tdp_pdl_wait();

    const int32_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    bool ok = true;
    if (warp == 0) {
        const uint32_t lead = at_rank(full, 0);
        uint32_t i = 0;
#pragma unroll 1
        for (int32_t t = first; t < a.tiles && ok; t += step) {
            const int32_t row = (t / a.tiles_c) * 256 + rank * 128, ch = (t % a.tiles_c) * 256 + rank * 128;
            // the second block has no channels where the tile has 128 or fewer
            const bool both = (t % a.tiles_c) * 256 + 128 < a.N, mine = rank == 0 || both;
            const uint32_t bytes = 2 * 16384 + (both ? 2 : 1) * (uint32_t)a.w_box * kK;
#pragma unroll 1
            for (int32_t k = 0; k < a.kb; ++k, ++i) {
                const uint32_t st = i % NST, to = base + st * SM::kStage;
                if (!(ok = mbar_wait(empty + 8 * st, ((i / NST) & 1) ^ 1, dead))) break;
                if (elect_one()) {
                    if (rank == 0) mbar_expect(full + 8 * st, bytes);       // both blocks' loads complete here
                    pair_load2(to, &map_x, lead + 8 * st, k * kK, row);
                    if (mine) pair_load2(to + 16384, &map_w, lead + 8 * st, k * kK, ch);
                }
                __syncwarp();
            }
        }
        // what has been loaded has been used, and so has landed
        for (uint32_t j = i > NST ? i - NST : 0; j < i; ++j) landed(empty + 8 * (j % NST), (j / NST) & 1);
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t id = idesc8(256, 256);
        uint32_t i = 0, n = 0;
#pragma unroll 1
        for (int32_t t = first; t < a.tiles && ok; t += step, ++n) {
            const uint32_t buf = n & 1;
            if (!(ok = mbar_wait(taken + 8 * buf, ((n >> 1) & 1) ^ 1, dead))) break;
            fence_after();
#pragma unroll 1
            for (int32_t k = 0; k < a.kb; ++k, ++i) {
                const uint32_t st = i % NST;
                if (!(ok = mbar_wait(full + 8 * st, (i / NST) & 1, dead))) break;
                fence_after();
                if (elect_one()) {
                    const uint32_t x = desc_rows(base + st * SM::kStage), w = desc_rows(base + st * SM::kStage + 16384);
#pragma unroll
                    for (int j = 0; j < 4; ++j) pair_mma8(tm + 256 * buf, x + 2 * j, w + 2 * j, id, k > 0 || j > 0);
                    pair_commit(empty + 8 * st);
                    if (k == a.kb - 1) pair_commit(sums + 8 * buf);
                }
                __syncwarp();
            }
        }
        if (elect_one()) pair_commit(drain);
        __syncwarp();
        landed(drain, 0);
    } else if (warp >= 4) {
        const int32_t r = threadIdx.x & 127, part = (warp - 4) >> 2;
        const uint32_t lanes = tm + ((uint32_t)(warp & 3) << 21) + 64 * part, to = out_s + (warp - 4) * SM::kOut;
        // A tile's scales and bias are asked for while the tile before is worked on.
        float x, w, b;
        auto ask = [&](int32_t t) {
            const int64_t row = (int64_t)(t / a.tiles_c) * 256 + rank * 128 + r;
            const int32_t ch = (t % a.tiles_c) * 256 + 64 * part + r;
            const bool in = r < 64 && ch < a.N;
            x = row < a.rows ? __ldcg(a.xs + row) : 1.f;
            w = in ? __ldcg(a.ws + ch) : 0.f;
            b = in && a.bias ? (float)static_cast<const T *>(a.bias)[ch] : 0.f;
        };
        if (first < a.tiles) ask(first);
        uint32_t n = 0, panel = 0;
        constexpr int W = BF16 ? 32 : 16;       // channels of a panel
        auto row_of = [&](int32_t t) { return (t / a.tiles_c) * 256 + (int32_t)rank * 128 + 32 * (warp & 3); };
        auto ch_of = [&](int32_t t) { return (t % a.tiles_c) * 256 + 64 * part; };
        // channels of a tile that this warp has: panels with anything in them are stored, each by the warp that filled it (by the
        // warpgroup, behind its barriers, 100000 x 64 x 1024 takes 57.6 us where this takes 54.4)
        auto end_of = [&](int32_t t) { return row_of(t) < a.rows ? min(64, a.N - ch_of(t)) : 0; };
        // The residual comes into the panel that its sum leaves by, a panel ahead: read by the threads, a row each, it took
        // 125 us where this takes 107 (35840 x 2048 x 2048).
        const uint32_t bars = added + 16 * (warp - 4);
        uint32_t phases = 0;
        bool asked = false;
        auto bring = [&](int32_t t, int32_t c0, uint32_t to_panel) {
            mbar_expect(bars + 8 * to_panel, 2048);
            tma_load2(to + to_panel * 2048, &map_r, bars + 8 * to_panel, ch_of(t) + c0, row_of(t));
        };
#pragma unroll 1
        for (int32_t t = first; t < a.tiles; t += step, ++n) {
            const uint32_t buf = n & 1;
            const int32_t row0 = row_of(t), ch0 = ch_of(t), end = end_of(t);
            const float xs = x;
            group_sync(1 + part);           // the last tile's have been read
            if (r < 64) {
                scales[64 * part + r] = w;
                scales[256 + 64 * part + r] = b;
            }
            if (t + step < a.tiles) ask(t + step);
            group_sync(1 + part);
            if (ok) ok = mbar_wait(sums + 8 * buf, (n >> 1) & 1, dead);
            ok = __all_sync(~0u, ok && !*dead);
            fence_after();
            const uint64_t x2 = ok ? pair(xs, xs) : pair(NAN, NAN);
            const bool far = __any_sync(~0u, !plain_scale(xs));
            auto take = [&] {
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(at_rank(taken + 8 * buf, 0));
            };
            if (end <= 0) take();
#pragma unroll 1
            for (int c0 = 0; c0 < end; c0 += W) {
                uint32_t v[W];
                if (BF16) tmem_ld32(lanes + 256 * buf + c0, v);
                else tmem_ld16(lanes + 256 * buf + c0, v);
                if (RES) {
                    const bool more = c0 + W < end;
                    const int32_t t2 = more ? t : t + step, c2 = more ? c0 + W : 0;
                    const bool next = more || (t2 < a.tiles && end_of(t2) > 0);
                    if (lane == 0) {
                        tma_store_read();       // both panels have left
                        if (!asked) bring(t, c0, panel);
                        if (next) bring(t2, c2, panel ^ 1);
                    }
                    asked = next;
                }
                tmem_wait_ld();
                if (BF16) tmem_have32(v);
                else tmem_have16(v);
                if (c0 + W >= end) take();
                if (RES) {
                    if (!mbar_wait(bars + 8 * panel, (phases >> panel) & 1, dead)) {
                        ok = false;
                        landed(bars + 8 * panel, (phases >> panel) & 1);
                    }
                    phases ^= 1u << panel;
                } else {
                    if (lane == 0) tma_store_read_but_one();    // the panel before the last has left
                    __syncwarp();
                }
                // (rows with far scales have a loop of their own: asked for at each value, 48862 x 448 x 4864 takes 204 us where this takes 177)
                auto sums_out = [&](auto any_far) {
                    constexpr bool FAR = decltype(any_far)::value;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t at = to + panel * 2048 + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4);        // the 64-byte swizzle of the maps
                        float f[E::kVec];
#pragma unroll
                        for (int q = 0; q < E::kVec; q += 4) {
                            const int c = 64 * part + c0 + j * E::kVec + q;
                            const ulonglong2 w4 = *reinterpret_cast<const ulonglong2 *>(scales + c), b4 = *reinterpret_cast<const ulonglong2 *>(scales + 256 + c);
                            const uint32_t *u = v + j * E::kVec + q;
                            unpair(fma2(mul2(pair(__uint_as_float(u[0]), __uint_as_float(u[1])), x2), w4.x, b4.x), f[q], f[q + 1]);
                            unpair(fma2(mul2(pair(__uint_as_float(u[2]), __uint_as_float(u[3])), x2), w4.y, b4.y), f[q + 2], f[q + 3]);
                            if (FAR && !plain_scale(xs)) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) f[q + i] = far_scaled(ok ? __uint_as_float(u[i]) : NAN, xs, scales[c + i], scales[256 + c + i]);
                            }
                        }
                        if (RES) {
                            float g[E::kVec];
                            uint4 s;
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(s.x), "=r"(s.y), "=r"(s.z), "=r"(s.w) : "r"(at) : "memory");
                            E::unpack(s, g);
#pragma unroll
                            for (int q = 0; q < E::kVec; ++q) f[q] = ok ? f[q] + g[q] : NAN;
                        }
                        const uint4 p = E::pack(f);
                        const uint32_t o[4] = {p.x, p.y, p.z, p.w};
                        st_shared16(at, o);
                    }
                };
                if (far) sums_out(std::true_type{});
                else sums_out(std::false_type{});
                fence_async();
                __syncwarp();
                if (lane == 0) tma_store2(&map_o, to + panel * 2048, ch0 + c0, row0);
                panel ^= 1;
            }
        }
        if (lane == 0) tma_store_done();
    }
    __syncwarp();
    fence_before();
    cluster_sync();         // neither block leaves, or frees its sums, while the other's products or arrivals may come
    if (warp == 2) pair_free(tm, 512);
}

}  // namespace tdp_m8

namespace {

using namespace tdp_m8;

// Map of e4m3 rows: boxes of 128 values by `box` rows in 128-byte-swizzled panels; zeros past the ends.
bool map8(CUtensorMap *map, const void *p, int64_t K, int64_t rows, int box)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = tdp_encode_tiled();
    if (!encode) return false;
    const cuuint64_t extent[2] = {(cuuint64_t)K, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)K};
    const cuuint32_t b[2] = {(cuuint32_t)kK, (cuuint32_t)box}, one[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), extent, stride, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of the outputs, or of the residual: boxes of 64 bytes by 32 rows.
bool map_out(CUtensorMap *map, void *p, int bf16, int64_t N, int64_t rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = tdp_encode_tiled();
    if (!encode) return false;
    const cuuint64_t extent[2] = {(cuuint64_t)N, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)N * (bf16 ? 2 : 4)};
    const cuuint32_t b[2] = {bf16 ? 32u : 16u, 32}, one[2] = {1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p, extent, stride, b, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A dependent launch of clusters of `size` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), unsigned grid, unsigned size, unsigned block, size_t smem, cudaStream_t s, Args &&...args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Parts of K of a tile: until the device has a block for every SM.
unsigned split_k(int64_t tiles, int32_t kb)
{
    unsigned split = 1;
    while (split < 8 && 2 * split <= (unsigned)kb && tiles * split < 152) split *= 2;
    return split;
}

template <int BF16, int NT>
cudaError_t tile_launch(args a, const void *w8, const void *x8, int64_t K, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    constexpr size_t bytes = tile_smem<NT>::kBytes;
    cudaError_t e = tdp_allow_smem(tdp_matmul8_tile_kernel<BF16, NT>, bytes, done);
    CUtensorMap w, x;
    a.w_box = std::min(128, a.N);
    a.x_box = (int32_t)std::min<int64_t>(NT, a.rows);
    if (e == cudaSuccess && (!map8(&w, w8, K, a.N, a.w_box) || !map8(&x, x8, K, a.rows, a.x_box))) e = cudaErrorInvalidValue;
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)a.tiles_c * ((a.rows + NT - 1) / NT);
    const unsigned split = split_k(tiles, a.kb);
    return launch_clusters(tdp_matmul8_tile_kernel<BF16, NT>, (unsigned)(tiles * split), split, kTileThreads, bytes, s, a, w, x);
}

template <int BF16, int RES>
cudaError_t pair_launch(args a, const void *w8, const void *x8, int64_t K, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    constexpr size_t bytes = pair_smem::kBytes;
    cudaError_t e = tdp_allow_smem(tdp_matmul8_pair_kernel<BF16, RES>, bytes, done);
    CUtensorMap w, x, o, r;
    a.w_box = std::min(128, a.N);
    a.x_box = 128;
    if (e == cudaSuccess && (!map8(&w, w8, K, a.N, a.w_box) || !map8(&x, x8, K, a.rows, a.x_box) || !map_out(&o, a.out, BF16, a.N, a.rows) ||
                             !map_out(&r, RES ? const_cast<void *>(a.res) : a.out, BF16, a.N, a.rows)))
        e = cudaErrorInvalidValue;
    if (e != cudaSuccess) return e;
    a.tiles_c = (a.N + 255) / 256;
    a.tiles = a.tiles_c * (int32_t)((a.rows + 255) / 256);
    return launch_clusters(tdp_matmul8_pair_kernel<BF16, RES>, 2 * std::min(a.tiles, 76), 2, kPairThreads, bytes, s, a, x, w, o, r);
}

// Rows of a tile, or 0 for pairs: the least time of the launch and of rounds of resident blocks, each so much for its end and for
// every stage of a block, in us as measured.  K = N = 2048, 16 / 128 / 512 / 1024 / 2048 rows: 3.9 / 5.3 / 13.1 / 24.7 / - by 16 rows,
// 4.5 / 5.2 / 7.3 / 14.0 / - by 32, 6.0 / 6.6 / 7.5 / 9.6 / - by 64, 8.8 / 9.3 / 9.5 / 9.8 / 10.6 by pairs; K = N = 4096: 4.7 / 9.9 / 37.7 /
// 70.6, 5.9 / 7.9 / 21.5 / 41.5, 8.5 / 7.9 / 13.7 / 26.2 and 13.0 / 13.6 / 14.0 / 15.3 / 24.0.  (Tiles of 128 rows were never best;
// eight stages in place of four, and so one block an SM, took 8.1 us where 32 rows take 5.2.)  Rows of K values that are no multiple of 128
// lie across lines, of 32 across sectors, which costs the smaller tiles more: 12982 x 128, K = 1280 / 1296 / 1312, takes 8.3 / 14.8 / 9.9 us by 64
// rows, x 136 by pairs 7.6 / 8.9 / 7.9.
int choose(int64_t rows, int32_t N, int64_t K, int32_t kb)
{
    const double across = K % 32 ? 1.9 : K % 128 ? 1.25 : 1.0, across2 = K % 32 ? 1.2 : 1.0;
    constexpr int nt[3] = {16, 32, 64};
    constexpr double end[3] = {2.3, 2.6, 3.4}, stage[3] = {0.20, 0.235, 0.285};
    double least = 5.0 + 0.275 * across2 * kb * (double)(((rows + 255) / 256 * ((N + 255) / 256) + 75) / 76);
    int best = 0;
    for (int i = 0; i < 3; ++i) {
        const int64_t tiles = (rows + nt[i] - 1) / nt[i] * ((N + 127) / 128), split = split_k(tiles, kb);
        const double cost = 1.0 + (end[i] + stage[i] * across * (double)((kb + split - 1) / split)) * (double)((tiles * split + 303) / 304);
        if (cost < least) {
            least = cost;
            best = nt[i];
        }
    }
    return best;
}

template <int BF16>
cudaError_t matmul8(const args &a, const void *w8, const void *x8, int64_t K, cudaStream_t s)
{
    switch (choose(a.rows, a.N, K, a.kb)) {
    case 16: return tile_launch<BF16, 16>(a, w8, x8, K, s);
    case 32: return tile_launch<BF16, 32>(a, w8, x8, K, s);
    case 64: return tile_launch<BF16, 64>(a, w8, x8, K, s);
    default: return a.res ? pair_launch<BF16, 1>(a, w8, x8, K, s) : pair_launch<BF16, 0>(a, w8, x8, K, s);
    }
}

}  // namespace

extern "C" tdp_status tdp_matmul8(tdp_plan_t plan, int64_t rows, int32_t K, int32_t N, const uint8_t *x8, const float *x8_scale,
                                  const uint8_t *w8, const float *w8_scale, const void *bias, const void *res, void *out,
                                  tdp_stream_t stream)
{
    if (!plan) return tdp_fail(TDP_ERR_INVALID_ARG, "null plan");
    const tdp_geom &g = plan->g;
    if (rows < 0 || K < 1 || N < 1) return tdp_fail(TDP_ERR_INVALID_ARG, "need rows >= 0, K >= 1 and N >= 1");
    if (K % 16 != 0 || (int64_t)N * g.esize % 16 != 0)
        return tdp_fail(TDP_ERR_MISALIGNED, "K and N * element size must be multiples of 16 bytes");
    if (K > TDP_MAX_MATMUL8 || N > TDP_MAX_MATMUL8 || rows > TDP_MAX_MATMUL8_ROWS)
        return tdp_fail(TDP_ERR_TOO_LARGE, "K or N above TDP_MAX_MATMUL8, or rows above TDP_MAX_MATMUL8_ROWS");
    if (rows == 0) return tdp_ok();
    if (!x8 || !x8_scale || !w8 || !w8_scale || !out) return tdp_fail(TDP_ERR_INVALID_ARG, "null x8, w8, scales or out");
    if (!tdp_aligned(x8, 16) || !tdp_aligned(w8, 16) || !tdp_aligned(bias, 16) || !tdp_aligned(res, 16) || !tdp_aligned(out, 16) ||
        !tdp_aligned(x8_scale, 4) || !tdp_aligned(w8_scale, 16))
        return tdp_fail(TDP_ERR_MISALIGNED, "rows, w8_scale and bias need 16-byte, x8_scale 4-byte alignment");
    if ((rows + 127) / 128 * ((N + 127) / 128) > (1 << 28)) return tdp_fail(TDP_ERR_TOO_LARGE, "rows * N above 2^42");
    const int64_t n = rows * N * g.esize;
    if (tdp_overlap(out, n, x8, rows * K) || tdp_overlap(out, n, w8, (int64_t)N * K) || tdp_partly(out, res, n))
        return tdp_fail(TDP_ERR_INVALID_ARG, "out over x8, w8 or a part of res");
    args a = {x8_scale, w8_scale, bias, res, out, rows, N, (K + kK - 1) / kK, (N + 127) / 128, 0, 0, 0};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = g.dtype == TDP_BF16 ? matmul8<1>(a, w8, x8, K, s) : matmul8<0>(a, w8, x8, K, s);
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}
