// tdp_xattn_tc.cuh -- bf16 cross attention on the tensor cores (tcgen05), forward.
//
// A block takes two tiles of 128 packed rows against the same key head and walks the kept
// 128-state tiles.  For tile t: S_t = Q_t K^T (tensor memory, fp32), p = exp2(c S_t - m) by one warpgroup,
// a row a thread, written back to tensor memory over S_t as bf16, O_t += P_t V.  While one tile's
// probabilities are computed the other tile's products run:
//   warps 0-3, 4-7   softmax of tile 0, 1 and its output
//   warp 8           loads Q, K and V tiles through tensor maps
//   warp 9           issues the products
//   warps 10, 11     zero the rows of V that a mask drops (their memory may hold anything, and 0 * NaN is not 0)
// The sums are rescaled only when a row's maximum has grown by more than 2^8 (p then stays below 2^8,
// exact in the fp32 sums and no coarser in bf16); the last scale divides out.  A persistent grid, one block
// per SM, takes (segment, part of the states, head block, row block) items in turn: the next item's loads
// and first products run under this one's output.
#pragma once

#include "tdp_tc.cuh"
#include "tdp_xattn.h"

namespace tdp_xt {

using namespace tdp_tc;

constexpr int kKeys = 128;              // states of a tile
constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;            // log2 by which a maximum may grow before the sums are rescaled

template <int DP>
struct fwd_smem {
    static constexpr int kTile = 128 * DP * 2;
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr int kBytes = 1024 + (2 + kStages) * kTile + 512;
};

// The kept state tiles of an item: with a mask, a list of tiles and of the masks of their states.
struct key_list {
    const int32_t *tile;
    const uint4 *words;
    int32_t n, j0, S;
    __device__ __forceinline__ int32_t at(int32_t j) const { return tile ? __ldg(tile + j) : j0 + j; }
    __device__ __forceinline__ uint4 mask(int32_t j) const
    {
        if (words) return __ldg(words + j);
        const int32_t left = S - (j0 + j) * kKeys;
        auto w = [&](int32_t o) { return left >= o + 32 ? ~0u : left <= o ? 0u : (1u << (left - o)) - 1u; };
        return make_uint4(w(0), w(32), w(64), w(96));
    }
};
__device__ __forceinline__ bool whole(const uint4 &m) { return (m.x & m.y & m.z & m.w) == ~0u; }

// One work item.
struct item {
    tdp_seg seg;
    int64_t tok0;                   // first token of the block in its segment
    int32_t left;                   // tokens of the segment from there on; <= 0: nothing to do
    int32_t head;                   // first query head
    int32_t kvh, part;
    key_list keys;
};

__device__ __forceinline__ item item_at(const tdp_geom &g, const xattn_args &a, int32_t w)
{
    item it;
    const int32_t blk = w % a.blocks, hb = a.Hq / a.Gp;
    w /= a.blocks;
    it.head = w % hb * a.Gp;
    it.kvh = it.head / a.G;
    w /= hb;
    it.part = w % a.split;
    it.seg = xattn_seg(g, a, w / a.split);
    it.tok0 = (int64_t)blk * 2 * a.TT;
    it.left = (int32_t)(it.seg.T - it.tok0);
    const int32_t tiles = (a.S + kKeys - 1) / kKeys;
    int32_t n = tiles;
    it.keys.S = a.S;
    it.keys.tile = nullptr;
    it.keys.words = nullptr;
    int64_t m = 0;
    if (a.mask) {
        m = a.per_tile ? (int64_t)it.seg.t * g.B + it.seg.b : it.seg.b;
        n = __ldg(a.kept_n + m);
    }
    const int32_t per = (n + a.split - 1) / a.split;
    it.keys.j0 = min(n, it.part * per);
    it.keys.n = min(n, it.keys.j0 + per) - it.keys.j0;
    if (a.mask) {
        it.keys.tile = a.kept_tile + m * tiles + it.keys.j0;
        it.keys.words = a.kept_words + m * tiles + it.keys.j0;
    }
    return it;
}

// Scores of the states that the mask word drops become -inf.
__device__ __forceinline__ void drop(uint32_t *s, uint32_t word)
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (!((word >> i) & 1)) s[i] = 0xff800000u;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
tdp_xattn_tc_kernel(const __grid_constant__ tdp_geom g, const __grid_constant__ xattn_args a,
                    const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, int32_t items)
{
    using SM = fwd_smem<DP>;
    using T = __nv_bfloat16;
    constexpr int NST = SM::kStages;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t q_s = base, kv_s = base + 2 * SM::kTile, bars = kv_s + NST * SM::kTile;
    const uint32_t full = bars, empty = full + 8 * NST, clean = empty + 8 * NST, qfull = clean + 8 * NST, qempty = qfull + 16,
                   sfull = qempty + 16, pfull = sfull + 16, odone = pfull + 16, drain = odone + 16;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_flag;
    volatile int *dead = &dead_flag;
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 9) tmem_alloc(smem_u32(&tmem_slot), 512);
    if (threadIdx.x == 0) {
        dead_flag = 0;
        for (int i = 0; i < NST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
            mbar_init(clean + 8 * i, 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(qfull + 8 * t, 1);
            mbar_init(qempty + 8 * t, 1);
            mbar_init(sfull + 8 * t, 1);
            mbar_init(pfull + 8 * t, 4);
            mbar_init(odone + 8 * t, 1);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = tmem_slot;
    tdp_pdl_trigger();
    tdp_pdl_wait();

    // registers: 168 a thread at launch, 504 for the three warps of a scheduler; 216 + 216 + 72 of them after
    if (warp >= 8) {
        regs_dec<72>();
        bool ok = true;
        uint32_t kv = 0;                        // K and V tiles so far: K and V take turns
        if (warp == 8 && lane == 0) {
            uint32_t qph = 0;
            constexpr uint32_t kTileBytes = SM::kTile;
            // a broadcast dimension (stride 0) is read at coordinate 0
            const int32_t k_heads = a.k_head > 0, v_heads = a.v_head > 0, k_items = a.k_item > 0, v_items = a.v_item > 0;
            const uint32_t q_bytes = (uint32_t)(a.Gp * a.TT) * DP * 2;
            for (int32_t w = blockIdx.x; w < items && ok; w += gridDim.x) {
                const item it = item_at(g, a, w);
                const int32_t n = it.keys.n, nt = it.left > a.TT ? 2 : 1;
                if (it.left <= 0 || n == 0) continue;
                auto load_q = [&](int t) {
                    ok = mbar_wait(qempty + 8 * t, ((qph >> t) & 1) ^ 1, dead);
                    if (!ok) return;
                    qph ^= 1u << t;
                    mbar_expect(qfull + 8 * t, q_bytes);
                    const int32_t row = (int32_t)(it.seg.row0 + it.tok0) + t * a.TT;
                    for (int p = 0; p < DP / 64; ++p)
                        tma_load3(q_s + t * SM::kTile + p * 16384, &map_q, qfull + 8 * t, 64 * p, it.head, row);
                };
                auto load_kv = [&](const CUtensorMap *map, int32_t tile) {
                    const uint32_t st = kv % NST;
                    ok = mbar_wait(empty + 8 * st, ((kv / NST) & 1) ^ 1, dead);
                    if (!ok) return;
                    ++kv;
                    mbar_expect(full + 8 * st, kTileBytes);
                    for (int p = 0; p < DP / 64; ++p)
                        tma_load4(kv_s + st * SM::kTile + p * 16384, map, full + 8 * st, 64 * p, map == &map_k ? it.kvh * k_heads : it.kvh * v_heads, tile * kKeys,
                                  map == &map_k ? it.seg.b * k_items : it.seg.b * v_items);
                };
                int32_t tile = it.keys.at(0);
                load_q(0);
                if (ok) load_kv(&map_k, tile);
                if (ok && nt == 2) load_q(1);
                for (int32_t j = 0; j < n && ok; ++j) {
                    const int32_t next = j + 1 < n ? it.keys.at(j + 1) : 0;
                    load_kv(&map_v, tile);
                    if (ok && j + 1 < n) load_kv(&map_k, next);
                    tile = next;
                }
            }
            // nothing may land after the block has gone: the last load into each stage and Q tile
            auto landed = [&](uint32_t bar, uint32_t parity) {
                for (uint32_t i = 0; i < kWaitRounds && !mbar_try(bar, parity); ++i) {
                }
            };
            for (uint32_t i = kv > NST ? kv - NST : 0; i < kv; ++i) landed(full + 8 * (i % NST), (i / NST) & 1);
            for (int t = 0; t < 2; ++t) landed(qfull + 8 * t, ((qph >> t) & 1) ^ 1);
        } else if (warp == 9 && lane == 0) {
            constexpr uint32_t id_pv = idesc(128, DP, false, true);
            const uint32_t id_qk = idesc(128, 128, false, false) | (a.scale < 0.f ? kNegateA : 0u);
            uint32_t qph = 0, pph = 0, cph = 0;     // phase of each tile's and stage's barrier
            auto qk = [&](int t, uint32_t st, bool last) {
                uint32_t x = desc_rows(q_s + t * SM::kTile), y = desc_rows(kv_s + st * SM::kTile);
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    mma_ss(tm + 128 * t, x, y, id_qk, i > 0);
                    const uint32_t d = i % 4 == 3 ? (16384 - 96) >> 4 : 2;      // next panel, or 32 bytes
                    x += d;
                    y += d;
                }
                mma_commit(sfull + 8 * t);
                if (last) mma_commit(qempty + 8 * t);
            };
            for (int32_t w = blockIdx.x; w < items && ok; w += gridDim.x) {
                const item it = item_at(g, a, w);
                const int32_t n = it.keys.n, nt = it.left > a.TT ? 2 : 1;
                if (it.left <= 0 || n == 0) continue;
                uint32_t st = kv % NST, ph = (kv / NST) & 1;
                bool dirty = a.mask && !whole(it.keys.mask(0));
                for (int t = 0; t < nt && ok; ++t) {
                    ok = mbar_wait(qfull + 8 * t, (qph >> t) & 1, dead);
                    qph ^= 1u << t;
                    if (ok && t == 0) ok = mbar_wait(full + 8 * st, ph, dead);
                    if (ok) qk(t, st, n == 1);
                }
                if (!ok) break;
                mma_commit(empty + 8 * st);
                for (int32_t j = 0; j < n && ok; ++j) {
                    const uint32_t v = kv + 2 * j + 1, vs = v % NST, ks = (v + 1) % NST;
                    ok = mbar_wait(full + 8 * vs, (v / NST) & 1, dead);
                    if (ok && dirty) {
                        ok = mbar_wait(clean + 8 * vs, (cph >> vs) & 1, dead);
                        cph ^= 1u << vs;
                    }
                    dirty = a.mask && j + 1 < n && !whole(it.keys.mask(j + 1));
                    for (int t = 0; t < nt && ok; ++t) {
                        ok = mbar_wait(pfull + 8 * t, (pph >> t) & 1, dead);
                        pph ^= 1u << t;
                        if (!ok) break;
                        fence_after();
                        const uint32_t y = desc_cols(kv_s + vs * SM::kTile, 16384);
#pragma unroll
                        for (int i = 0; i < kKeys / 16; ++i)
                            mma_ts(tm + 256 + DP * t, tm + 128 * t + 8 * i, y + i * (2048 >> 4), id_pv, j > 0 || i > 0);
                        mma_commit(odone + 8 * t);
                        if (j + 1 < n) {
                            if (t == 0) ok = mbar_wait(full + 8 * ks, ((v + 1) / NST) & 1, dead);
                            if (ok) qk(t, ks, j + 2 == n);
                        }
                    }
                    if (!ok) break;
                    mma_commit(empty + 8 * vs);
                    if (j + 1 < n) mma_commit(empty + 8 * ks);
                }
                kv += 2 * n;
            }
            mma_commit(drain);
            for (uint32_t i = 0; i < kWaitRounds && !mbar_try(drain, 0); ++i) {
            }
        } else if (warp >= 10 && a.mask) {
            const int32_t tid = threadIdx.x - 320;
            for (int32_t w = blockIdx.x; w < items && ok; w += gridDim.x) {
                const item it = item_at(g, a, w);
                if (it.left <= 0) continue;
                for (int32_t j = 0; j < it.keys.n && ok; ++j) {
                    const uint4 m = it.keys.mask(j);
                    if (whole(m)) continue;
                    const uint32_t v = kv + 2 * j + 1, st = v % NST;
                    ok = mbar_wait(full + 8 * st, (v / NST) & 1, dead);
                    if (!ok) break;
                    constexpr int C = DP / 8;           // 16-byte chunks of a row
                    for (int32_t i = tid; i < 128 * C; i += 64) {
                        const int32_t r = i / C, c = i % C;
                        const uint32_t word = r < 64 ? (r < 32 ? m.x : m.y) : (r < 96 ? m.z : m.w);
                        if (!((word >> (r & 31)) & 1))
                            st_zero16(kv_s + st * SM::kTile + (c / 8) * 16384 + panel_off(r, c & 7));
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(clean + 8 * st);
                }
                kv += 2 * it.keys.n;
            }
        }
        __syncwarp();
    } else {
        regs_inc<216>();
        const int32_t t = warp >> 2;
        const uint32_t lanes = tm + ((uint32_t)(warp & 3) << 21);      // this warp's 32 lanes
        const uint32_t S = lanes + 128 * t, O = lanes + 256 + DP * t;
        // a scale of zero weighs every state alike, and so does one too small to matter; -inf stays -inf
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
        const int32_t r = 32 * (warp & 3) + lane, rt = r / a.Gp, rh = r - rt * a.Gp;      // this row's token and head
        uint32_t sn = 0, on = 0;
        bool ok = true;
        for (int32_t w = blockIdx.x; w < items; w += gridDim.x) {
            const item it = item_at(g, a, w);
            const int32_t n = it.keys.n;
            if (it.left <= t * a.TT) continue;
            const bool mine = rt < a.TT && t * a.TT + rt < it.left;
            const bool warp_on = __any_sync(~0u, mine);
            float m = -INFINITY, l = 0.f;
            for (int32_t j = 0; j < n && ok; ++j) {
                const uint4 mk = it.keys.mask(j);
                ok = mbar_wait(sfull + 8 * t, sn & 1, dead);
                ++sn;
                if (!ok) break;
                fence_after();
                if (warp_on) {
                    uint32_t s[128];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld32(S + 32 * i, s + 32 * i);
                    tmem_wait_ld();
                    if (!whole(mk)) {
                        drop(s, mk.x);
                        drop(s + 32, mk.y);
                        drop(s + 64, mk.z);
                        drop(s + 96, mk.w);
                    }
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 128; i += 8)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            top[u] = fmaxf(top[u], fmaxf(__uint_as_float(s[i + u]), __uint_as_float(s[i + 4 + u])));
                    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
                    const bool grow = mx > m + kGrow;       // true for the first kept state: m = -inf
                    if (__any_sync(~0u, grow)) {
                        const float mn = grow ? mx : m, f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
                        l *= f;
                        m = mn;
                        if (j > 0) {
                            ok = mbar_wait(odone + 8 * t, on & 1, dead);
                            fence_after();
#pragma unroll 1
                            for (int i = 0; i < DP / 16; ++i) {
                                uint32_t o[16];
                                tmem_ld16(O + 16 * i, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                                tmem_st16(O + 16 * i, o);
                            }
                        }
                    }
                    const float b = m == -INFINITY ? 0.f : -m;
                    const uint64_t c2 = pair(c, c), b2 = pair(b, b);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t p[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            float x, y;
                            unpair(fma2(pair(__uint_as_float(s[32 * i + 2 * u]), __uint_as_float(s[32 * i + 2 * u + 1])), c2, b2), x, y);
                            x = exp2_fast(x);
                            y = exp2_fast(y);
                            sum[u & 1] = add2(sum[u & 1], pair(x, y));
                            p[u] = tdp_pack_bf16x2(x, y);
                        }
                        tmem_st16(S + 16 * i, p);
                    }
                    float x, y;
                    unpair(add2(sum[0], sum[1]), x, y);
                    l += x + y;
                    tmem_wait_st();
                }
                if (j > 0) ++on;
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + 8 * t);
            }
            // output: O / l, or zero where nothing is kept, or NaN after a lost wait
            if (n > 0 && ok) {
                ok = mbar_wait(odone + 8 * t, on & 1, dead);
                ++on;
                fence_after();
            }
            const int64_t h = (it.seg.row0 + it.tok0 + t * a.TT + rt) * a.Hq + it.head + rh;
            const float inv = !ok ? NAN : l == 0.f ? 0.f : 1.f / l;
            if (warp_on) {
                const int64_t all = (int64_t)it.part * a.rows * a.Hq + h;
#pragma unroll
                for (int i = 0; i < DP / 32; ++i) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32(O + 32 * i, o);
                        tmem_wait_ld();
                    }
                    // without a kept state O holds nothing
#pragma unroll
                    for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(inv == 0.f ? 0.f : __uint_as_float(o[u]) * inv);
                    if (mine && a.split > 1) {
                        float *dst = a.po + all * a.D + 32 * i;
#pragma unroll
                        for (int u = 0; u < 32; u += 8)
                            if (32 * i + u < a.D) st_global32(dst + u, o + u);
                    } else if (mine) {
                        T *dst = static_cast<T *>(a.out) + h * a.D + 32 * i;
                        uint32_t b[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u) b[u] = tdp_pack_bf16x2(__uint_as_float(o[2 * u]), __uint_as_float(o[2 * u + 1]));
                        if (a.D % 16 == 0) {        // whole 32-byte sectors
#pragma unroll
                            for (int u = 0; u < 16; u += 8)
                                if (32 * i + 2 * u < a.D) st_global32(dst + 2 * u, b + u);
                        } else {
#pragma unroll
                            for (int u = 0; u < 16; u += 4)
                                if (32 * i + 2 * u < a.D) *reinterpret_cast<uint4 *>(dst + 2 * u) = make_uint4(b[u], b[u + 1], b[u + 2], b[u + 3]);
                        }
                    }
                    __syncwarp();
                }
                const float lse = !ok ? NAN : l == 0.f ? -INFINITY : m * kLn2 + logf(l);
                if (mine && a.split > 1) a.pl[all] = lse;
                else if (mine && a.lse) a.lse[h] = lse;
            }
            fence_before();
        }
    }
    __syncthreads();
    if (warp == 9) tmem_free(tm, 512);
}

// One block per mask row: the 128-state tiles that keep a state, in order, and their masks.
__global__ void __launch_bounds__(1024)
tdp_xattn_kept_kernel(const uint8_t *mask, int32_t S, int32_t *kept_n, int32_t *kept_tile, uint4 *kept_words)
{
    __shared__ uint32_t found[2][32];
    const int32_t tiles = (S + kKeys - 1) / kKeys, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const uint8_t *m = mask + row * S;
    const int32_t warps = blockDim.x >> 5;
    int32_t n = 0;
    for (int32_t t0 = 0, odd = 0; t0 < tiles; t0 += warps, odd ^= 1) {
        const int32_t t = t0 + warp;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t s = t * kKeys + 32 * i + lane;
            w[i] = __ballot_sync(~0u, t < tiles && s < S && m[s] != 0);
        }
        const bool any = (w[0] | w[1] | w[2] | w[3]) != 0;
        if (lane == 0) found[odd][warp] = any;
        __syncthreads();
        const uint32_t all = __ballot_sync(~0u, lane < warps && found[odd][lane] != 0);
        if (any && lane == 0) {
            const int64_t at = row * tiles + n + __popc(all & ((1u << warp) - 1u));
            kept_tile[at] = t;
            kept_words[at] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        n += __popc(all);
    }
    if (threadIdx.x == 0) kept_n[row] = n;
}

}  // namespace tdp_xt
