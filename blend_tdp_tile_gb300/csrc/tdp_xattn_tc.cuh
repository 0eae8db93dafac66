// tdp_xattn_tc.cuh -- bf16 cross attention on the tensor cores (tcgen05), forward.
//
// A block takes two tiles of 128 packed rows against the same key head and walks the kept
// 128-state tiles.  For tile t: S_t = Q_t K^T (tensor memory, fp32), p = exp2(c S_t - m) by one warpgroup,
// a row a thread, written back to tensor memory over S_t as bf16, O_t += P_t V.  While one tile's
// probabilities are computed the other tile's products run; scores are made two or three (kScores) tiles ahead:
//   warps 0-3, 4-7   softmax of tile 0, 1 and its output
//   warp 8, 10       load K and V tiles, Q tiles, through tensor maps
//   warp 9           issues the products; P V starts when half of the probabilities are there
//   warp 11          zeroes the rows of V that a mask drops (their memory may hold anything, and 0 * NaN is not 0)
// The sums are rescaled only when a row's maximum has grown by more than 2^8 (p then stays below 2^8,
// exact in the fp32 sums and no coarser in bf16); the last scale divides out.  p is rounded to bf16, as the tensor cores
// take it beside V's bf16: a relative 2^-8 at most, no more than V's own rounding; l sums p as it was before.  A persistent grid, one block
// per SM, takes (segment, part of the states, head block, row block) items in turn: the next item's loads
// and first products run under this one's output.
//
// Bound by the products at 128 columns a head: 35840 rows, 16 heads on 4, 640 states take 135 us (1.39 PFLOP/s, tensor
// pipe 58 % busy), 168960 rows of 16 heads against 512 states 540 us, the clock down to some 1.8 GHz at the card's
// power limit.  At 64 columns bound by the softmax and by the products with V, whose 64 columns take 54 cycles a step for
// 32 at the full rate: 16 heads, 1000 states 156 us (0.94 PFLOP/s).  One token an item is bound by the states' bytes: eight
// items, 32 heads on 8, 5760 kept states: 36 us, 5.2 TB/s.
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
    // even: a stage always holds K or always V, so that the cleaning warp, which waits for V tiles alone, meets every
    // phase of their stages' barriers (a wait for a phase two ahead returns at once)
    static constexpr int kStages = DP == 128 ? 4 : 8;
    // Buffers of scores in tensor memory, beside the outputs.  The third lets a tile's next scores be made while its
    // softmax works: 64 columns a head are bound by the softmax, not by the products.
    static constexpr int kScores = DP == 128 ? 2 : 3;
    static constexpr int kOut = 16384;          // a panel of outputs on its way to memory, per tile
    static constexpr int kBytes = 1024 + (2 + kStages) * kTile + 2 * kOut + 512;
};

// Number of this warp's role: 0-7 are the hardware's warps 4-11, 8-11 its warps 0-3.  The warps that issue products
// and loads come first because a scheduler prefers its oldest warps; behind the softmax's they waited for issue slots.
__device__ __forceinline__ int32_t role()
{
    const int32_t w = warp_id();
    return w < 4 ? w + 8 : w - 4;
}

// A place in a ring of N stages and the phase of its barriers.
template <int N>
struct ring {
    uint32_t st, ph;
    __device__ __forceinline__ void next()
    {
        if (++st == N) {
            st = 0;
            ph ^= 1;
        }
    }
    __device__ __forceinline__ void advance(uint32_t k)
    {
        const uint32_t to = st + k, rounds = to / N;
        st = to - rounds * N;
        ph ^= rounds & 1;
    }
};

// The kept state tiles of an item: with a mask, a list of tiles and of the masks of their states.  The kernel before writes
// the lists while this one is already resident: plain loads, which see it after the wait, not those for memory that never
// changes.  (By L2, a load a tile: both gradients at 16 heads of 64, 1000 states all kept by a mask, 561 us where this takes 527.)
struct key_list {
    const int32_t *tile;
    const uint4 *words;
    int32_t n, j0, S;
    __device__ __forceinline__ int32_t at(int32_t j) const { return tile ? tile[j] : j0 + j; }
    __device__ __forceinline__ uint4 mask(int32_t j) const
    {
        if (words) return words[j];
        const int32_t left = S - (j0 + j) * kKeys;
        auto w = [&](int32_t o) { return left >= o + 32 ? ~0u : left <= o ? 0u : (1u << (left - o)) - 1u; };
        return make_uint4(w(0), w(32), w(64), w(96));
    }
};
__device__ __forceinline__ bool whole(const uint4 &m) { return (m.x & m.y & m.z & m.w) == ~0u; }

// Zeroes the rows of a tile whose states are dropped, two or four rows at a time: a warp.  (Row by row with a test each
// took longer than the tile's products.)
template <int DP>
__device__ __forceinline__ void zero_dropped(uint32_t tile, const uint4 &m, int32_t lane)
{
    constexpr int C = DP / 8, R = 32 / C;       // 16-byte chunks of a row, rows at a time
    const int32_t col = lane % C;
#pragma unroll 1
    for (int32_t i = 0; i < 4; ++i) {
        uint32_t gone = ~(i < 2 ? (i ? m.y : m.x) : (i > 2 ? m.w : m.z));
#pragma unroll 1
        while (gone) {
            int32_t row = -1;
#pragma unroll
            for (int p = 0; p < R; ++p) {
                const int32_t r = __ffs(gone) - 1;
                gone &= gone - 1;
                if (lane / C == p) row = r;
            }
            if (row >= 0) st_zero16(tile + (col / 8) * 16384 + panel_off(32 * i + row, col & 7));
        }
    }
}

// One work item.
struct item {
    tdp_seg seg;
    int64_t tok0;                   // first token of the block in its segment
    int32_t left;                   // tokens of the segment from there on; <= 0: nothing to do
    int32_t head;                   // first query head
    int32_t kvh, part;
    int32_t rounds;                 // dq: walks over the kept state tiles, one or two, times their number
    key_list keys;
};

__device__ __forceinline__ item item_at(const tdp_geom &g, const xattn_args &a, int32_t w)
{
    item it;
    const int32_t blk = a.by_blocks.mod(w);
    it.head = a.by_heads.mod(w) * a.Gp;
    it.kvh = a.by_group.div(it.head);
    it.part = a.by_split.mod(w);
    it.seg = xattn_seg_fast(g, a, w);
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
        n = a.kept_n[m];
    }
    const int32_t per = a.by_split.div(n + a.split - 1);
    it.keys.j0 = min(n, it.part * per);
    it.keys.n = min(n, it.keys.j0 + per) - it.keys.j0;
    if (a.mask) {
        it.keys.tile = a.kept_tile + m * tiles + it.keys.j0;
        it.keys.words = a.kept_words + m * tiles + it.keys.j0;
    }
    return it;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
tdp_xattn_tc_kernel(const __grid_constant__ tdp_geom g, const __grid_constant__ xattn_args a,
                    const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, int32_t items)
{
    using SM = fwd_smem<DP>;
    using T = __nv_bfloat16;
    constexpr int NST = SM::kStages, NB = SM::kScores;
    constexpr uint32_t kO = NB * 128;           // first column of the outputs
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t q_s = base, kv_s = base + 2 * SM::kTile, out_s = kv_s + NST * SM::kTile,
                   bars = out_s + 2 * SM::kOut;
    const uint32_t full = bars, empty = full + 8 * NST, clean = empty + 8 * NST, qfull = clean + 8 * NST, qempty = qfull + 16,
                   sfull = qempty + 16, phalf = sfull + 32, pfull = phalf + 8 * NB, odone = pfull + 8 * NB, drain = odone + 32;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_flag;
    volatile int *dead = &dead_flag;
    const int32_t warp = role(), lane = threadIdx.x & 31;
    if (warp == 9) tmem_alloc(smem_u32(&tmem_slot), 512);
    if (threadIdx.x == 0) {
        dead_flag = 0;
        for (int i = 0; i < NST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
            mbar_init(clean + 8 * i, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(qfull + 8 * t, 1);
            mbar_init(qempty + 8 * t, 1);
            for (int b = 0; b < 16; b += 8) {
                mbar_init(sfull + 16 * t + b, 1);
                mbar_init(odone + 16 * t + b, 1);
            }
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(phalf + 8 * b, 4);
            mbar_init(pfull + 8 * b, 4);
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

    // The products, loads and cleaning share one loop over the items, so that the code holds each piece once: past
    // the instruction cache every step of a role cost some 350 cycles.  Registers: 168 a thread at launch, 504
    // for the three warps of a scheduler; 216 + 216 + 72 of them from here on.
    bool ok = true;
    uint32_t kv = 0;                        // K and V tiles so far: K and V take turns
    uint32_t ph = 0, ph2 = 0;               // phases of this role's barriers, a bit each (softmax: score tiles so far)
    if (warp < 8) {
        regs_inc<216>();
        const int32_t t = warp >> 2;            // tile
        const uint32_t lanes = tm + ((uint32_t)(warp & 3) << 21), O = lanes + kO + DP * t;       // this warp's lanes
        ring<NB> scores = {0, 0};               // buffer of the item's first scores
        // a scale of zero weighs every state alike, and so does one too small to matter; -inf stays -inf
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
        const int32_t r = threadIdx.x & 127, rt = r / a.Gp, rh = r - rt * a.Gp;         // row, its token and head
        // A tile's scores and its P V have two barriers each, in turn.  The next scores may be there before these are looked
        // at, and the products of the last step may still run: scores say that the products two steps back are done.
        auto products = [&](uint32_t i) { return mbar_wait(odone + 16 * t + 8 * (i & 1), (i >> 1) & 1, dead); };
        for (int32_t w = blockIdx.x; w < items; w += gridDim.x) {
            const item it = item_at(g, a, w);
            const int32_t n = it.keys.n;
            const uint32_t nt = it.left > a.TT ? 2 : it.left > 0 ? 1 : 0;
            ring<NB> cur = scores;
            scores.advance(n * nt);
            if ((uint32_t)t >= nt) continue;
            if (t == 1) cur.next();
            const bool mine = rt < a.TT && t * a.TT + rt < it.left;
            const bool warp_on = __any_sync(~0u, mine);
            const bool by_map = a.split == 1 && it.left - t * a.TT >= a.TT;
            const int32_t row0 = (int32_t)(it.seg.row0 + it.tok0) + t * a.TT, head = it.head, part = it.part;
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int32_t j = 0; j < n && ok; ++j) {
                const uint4 mk = it.keys.mask(j);
                const uint32_t S = lanes + 128 * cur.st, half = phalf + 8 * cur.st, whole_p = pfull + 8 * cur.st;
                ok = mbar_wait(sfull + 16 * t + 8 * (ph & 1), (ph >> 1) & 1, dead);
                if (!ok) break;
                ++ph;
                cur.advance(nt);
                fence_after();
                if (warp_on) {
                    uint32_t s[64], z[64];
                    tmem_ld32(S, s);
                    tmem_ld32(S + 32, s + 32);
                    tmem_ld32(S + 64, z);
                    tmem_ld32(S + 96, z + 32);
                    tmem_wait_ld();
                    tmem_have32(s);
                    tmem_have32(s + 32);
                    tmem_have32(z);
                    tmem_have32(z + 32);
                    if (!whole(mk)) {
                        // states that the mask drops
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            if (!((mk.x >> u) & 1)) s[u] = 0xff800000u;
                            if (!((mk.y >> u) & 1)) s[32 + u] = 0xff800000u;
                            if (!((mk.z >> u) & 1)) z[u] = 0xff800000u;
                            if (!((mk.w >> u) & 1)) z[32 + u] = 0xff800000u;
                        }
                    }
                    float top[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) top[u] = fmaxf(__uint_as_float(z[u]), __uint_as_float(s[u]));
#pragma unroll
                    for (int i = 4; i < 64; i += 4)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            top[u] = fmaxf(top[u], fmaxf(__uint_as_float(z[i + u]), __uint_as_float(s[i + u])));
                    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
                    const bool grow = mx > m + kGrow;       // true for the first kept state: m = -inf
                    if (__any_sync(~0u, grow)) {
                        const float mn = grow ? mx : m, f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
                        l *= f;
                        m = mn;
                        if (j > 0) {
                            ok = products(ph - 2);
                            fence_after();
#pragma unroll 1
                            for (int i = 0; i < DP / 16; ++i) {
                                uint32_t o[16];
                                tmem_ld16(O + 16 * i, o);
                                tmem_wait_ld();
                                tmem_have16(o);
#pragma unroll
                                for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                                tmem_st16(O + 16 * i, o);
                            }
                        }
                    }
                    const float b = m == -INFINITY ? 0.f : -m;
                    const uint64_t c2 = pair(c, c), b2 = pair(b, b);
                    uint64_t sum[2] = {0, 0};
                    auto exp32 = [&](const uint32_t *x32, int i) {
                        uint32_t p[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            float x, y;
                            unpair(fma2(pair(__uint_as_float(x32[2 * u]), __uint_as_float(x32[2 * u + 1])), c2, b2), x, y);
                            x = exp2_fast(x);
                            y = exp2_fast(y);
                            sum[u & 1] = add2(sum[u & 1], pair(x, y));
                            p[u] = tdp_pack_bf16x2(x, y);
                        }
                        tmem_st16(S + 16 * i, p);
                    };
                    exp32(s, 0);
                    exp32(s + 32, 1);
                    tmem_wait_st();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(half);
                    exp32(z, 2);
                    exp32(z + 32, 3);
                    float x, y;
                    unpair(add2(sum[0], sum[1]), x, y);
                    l += x + y;
                    tmem_wait_st();
                } else if (lane == 0) {
                    mbar_arrive(half);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(whole_p);
            }
            // output: O / l, or zero where nothing is kept, or NaN after a wait that any thread has lost
            if (n > 0 && ok) {
                ok = products(ph - 1);
                fence_after();
            }
            const int32_t h = (row0 + rt) * a.Hq + head + rh;
            const int64_t all = (int64_t)part * a.rows * a.Hq + h;
            ok = __all_sync(~0u, ok && !*dead);
            const float inv = !ok ? NAN : l == 0.f ? 0.f : 1.f / l;
            const float lse = !ok ? NAN : l == 0.f ? -INFINITY : m * kLn2 + logf(l);
            if (mine && a.split > 1) a.pl[all] = lse;
            else if (mine && a.lse) a.lse[h] = lse;
            // a whole tile leaves through shared memory: row by row from the threads, each sector of a store is
            // a line of its own to the load-store unit, 2000 cycles for the two tiles
            const uint32_t buf = out_s + t * SM::kOut;
            const bool issuer = r == 0;
#pragma unroll 1
            for (int i = 0; i < DP / 32; ++i) {
                uint32_t o[32], b[16];
                if (n > 0) {
                    tmem_ld32(O + 32 * i, o);
                    tmem_wait_ld();
                    tmem_have32(o);
                }
                // without a kept state O holds nothing
#pragma unroll
                for (int u = 0; u < 32; ++u) o[u] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(o[u]) * inv);
#pragma unroll
                for (int u = 0; u < 16; ++u) b[u] = tdp_pack_bf16x2(__uint_as_float(o[2 * u]), __uint_as_float(o[2 * u + 1]));
                if (by_map) {
                    if ((i & 1) == 0) {
                        if (issuer) tma_store_read();       // the buffer's last panel has left
                        group_sync(1 + t);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) st_shared16(buf + panel_off(r, 4 * (i & 1) + u), b + 4 * u);
                    if (i & 1) {
                        fence_async();
                        group_sync(1 + t);
                        if (issuer) tma_store3(&map_o, buf, 32 * (i - 1), head, row0);
                    }
                } else if (mine && a.split > 1) {
                    float *dst = a.po + all * a.D + 32 * i;
#pragma unroll
                    for (int u = 0; u < 32; u += 8)
                        if (32 * i + u < a.D) st_global32(dst + u, o + u);
                } else if (mine) {
                    T *dst = static_cast<T *>(a.out) + (int64_t)h * a.D + 32 * i;
#pragma unroll
                    for (int u = 0; u < 16; u += 4)
                        if (32 * i + 2 * u < a.D) *reinterpret_cast<uint4 *>(dst + 2 * u) = make_uint4(b[u], b[u + 1], b[u + 2], b[u + 3]);
                }
                __syncwarp();
            }
            fence_before();
        }
        if (r == 0) tma_store_done();
    } else {
        regs_dec<72>();
        ring<NB> made = {0, 0}, used = {0, 0};      // products: buffers of scores to be made and used
        for (int32_t w = blockIdx.x; w < items; w += gridDim.x) {
            const item it = item_at(g, a, w);
            const int32_t n = it.keys.n, nt = it.left > a.TT ? 2 : 1;
            if (it.left <= 0 || n == 0 || !ok) continue;
            if (warp == 8) {
                // a broadcast dimension (stride 0) is read at coordinate 0
#pragma unroll 1
                for (int32_t i = 0; i < 2 * n; ++i) {
                    const bool v = i & 1;
                    const uint32_t st = kv % NST;
                    const int32_t head = (v ? a.v_head : a.k_head) > 0 ? it.kvh : 0, b = (v ? a.v_item : a.k_item) > 0 ? it.seg.b : 0;
                    const int32_t state = it.keys.at(i >> 1) * kKeys;
                    if (!(ok = mbar_wait(empty + 8 * st, ((kv / NST) & 1) ^ 1, dead))) break;
                    ++kv;
                    if (elect_one()) {
                        mbar_expect(full + 8 * st, SM::kTile);
                        for (int p = 0; p < DP / 64; ++p)
                            tma_load4(kv_s + st * SM::kTile + p * 16384, v ? &map_v : &map_k, full + 8 * st, 64 * p, head, state, b);
                    }
                    __syncwarp();
                }
            } else if (warp == 10) {
#pragma unroll 1
                for (int q = 0; q < nt; ++q) {
                    if (!(ok = mbar_wait(qempty + 8 * q, ((ph >> q) & 1) ^ 1, dead))) break;
                    ph ^= 1u << q;
                    if (elect_one()) {
                        mbar_expect(qfull + 8 * q, (uint32_t)(a.Gp * a.TT) * DP * 2);
                        const int32_t row = (int32_t)(it.seg.row0 + it.tok0) + q * a.TT;
                        for (int p = 0; p < DP / 64; ++p)
                            tma_load3(q_s + q * SM::kTile + p * 16384, &map_q, qfull + 8 * q, 64 * p, it.head, row);
                    }
                    __syncwarp();
                }
            } else if (warp == 9) {
                constexpr uint32_t id_pv = idesc(128, DP, false, true);
                const uint32_t id_qk = idesc(128, 128, false, false) | (a.scale < 0.f ? kNegateA : 0u);
                // Steps i: row tile i % nt, state tile i / nt.  Scores are `look` steps ahead: P V of step i frees the buffer of the
                // scores of step i + look.  (One row tile looks two ahead at most: its softmax then knows that the products of the
                // step before last are done.)  The tensor cores queue two products, some 128 cycles, and a wait takes longer: the
                // next barrier is looked at before the last two are issued.
                const int32_t total = n * nt, look = nt == 2 ? NB : 2;
                bool there = false;
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    if (!there) ok = ok && mbar_wait(bar, parity, dead);
                    there = false;
                    __syncwarp();
                    return ok;
                };
                auto stage = [&](uint32_t i) { return i % NST; };
                auto phase = [&](uint32_t i) { return (i / NST) & 1; };
                const uint32_t v_full = a.mask ? clean : full;
                auto scores = [&](int32_t i) {
                    const int32_t q = nt == 2 ? i & 1 : 0, j = nt == 2 ? i >> 1 : i;
                    const uint32_t at = kv + 2 * j, s_t = tm + 128 * made.st;
                    if (j == 0) {
                        if (!(ok = ok && mbar_wait(qfull + 8 * q, (ph >> q) & 1, dead))) return;
                        ph ^= 1u << q;
                    }
                    if (q == 0 && !wait(full + 8 * stage(at), phase(at))) return;
                    const uint32_t x = desc_rows(q_s + q * SM::kTile), y = desc_rows(kv_s + stage(at) * SM::kTile);
                    auto step = [&](int k) {
                        const uint32_t o = (k / 4) * (16384 >> 4) + (k % 4) * 2;       // next panel, or 32 bytes
                        mma_ss(s_t, x + o, y + o, id_qk, k > 0);
                    };
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < DP / 16 - 2; ++k) step(k);
                    }
                    there = mbar_test(phalf + 8 * used.st, used.ph);       // the next step's probabilities
                    __syncwarp();
                    if (elect_one()) {
                        step(DP / 16 - 2);
                        step(DP / 16 - 1);
                        mma_commit(sfull + 16 * q + 8 * ((ph2 >> q) & 1));
                        if (q == nt - 1) mma_commit(empty + 8 * stage(at));
                        if (j == n - 1) mma_commit(qempty + 8 * q);
                    }
                    __syncwarp();
                    ph2 ^= 1u << q;
                    made.next();
                };
                for (int32_t i = 0; i < look && i < total && ok; ++i) {
                    scores(i);
                    there = false;
                }
#pragma unroll 1
                for (int32_t i = 0; i < total && ok; ++i) {
                    const int32_t q = nt == 2 ? i & 1 : 0, j = nt == 2 ? i >> 1 : i;
                    const uint32_t at = kv + 2 * j + 1, half = phalf + 8 * used.st, whole_p = pfull + 8 * used.st, p_ph = used.ph;
                    const uint32_t y = desc_cols(kv_s + stage(at) * SM::kTile, 16384), d = tm + kO + DP * q, p = tm + 128 * used.st;
                    if (q == 0 && !(ok = mbar_wait(v_full + 8 * stage(at), phase(at), dead))) break;
                    if (!wait(half, p_ph)) break;
                    fence_after();
                    auto step = [&](int k) { mma_ts(d, p + 8 * k, y + k * (2048 >> 4), id_pv, j > 0 || k > 0); };
                    if (elect_one()) {
                        step(0);
                        step(1);
                    }
                    there = mbar_test(whole_p, p_ph);
                    __syncwarp();
                    if (elect_one()) {
                        step(2);
                        step(3);
                    }
                    __syncwarp();
                    if (!wait(whole_p, p_ph)) break;
                    fence_after();
                    if (elect_one()) {
                        step(4);
                        step(5);
                    }
                    const uint32_t next_k = kv + 2 * ((i + look) / nt);
                    there = i + look < total && (nt == 1 || (i + look) % 2 == 0) && mbar_test(full + 8 * stage(next_k), phase(next_k));
                    __syncwarp();
                    if (elect_one()) {
                        step(6);
                        step(7);
                        mma_commit(odone + 16 * q + 8 * ((ph2 >> (2 + q)) & 1));
                        if (q == nt - 1) mma_commit(empty + 8 * stage(at));
                    }
                    __syncwarp();
                    ph2 ^= 4u << q;
                    used.next();
                    if (i + look < total) scores(i + look);
                    else there = false;
                }
                kv += 2 * n;
            } else if (warp == 11 && a.mask) {
#pragma unroll 1
                for (int32_t j = 0; j < n && ok; ++j) {
                    const uint4 m = it.keys.mask(j);
                    const uint32_t v = kv + 2 * j + 1, st = v % NST;
                    ok = mbar_wait(full + 8 * st, (v / NST) & 1, dead);
                    if (!ok) break;
                    zero_dropped<DP>(kv_s + st * SM::kTile, m, lane);
                    fence_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(clean + 8 * st);
                }
                kv += 2 * n;
            }
        }
    }
    // nothing may land, or be on its way, after the block has gone
    auto landed = [&](uint32_t bar, uint32_t parity) {
#pragma unroll 1
        for (uint32_t i = 0; i < kWaitRounds && !mbar_try(bar, parity); ++i) {
        }
    };
    if (warp >= 8) {
        if (warp == 8)
            for (uint32_t i = kv > NST ? kv - NST : 0; i < kv; ++i) landed(full + 8 * (i % NST), (i / NST) & 1);
        if (warp == 10)
            for (int q = 0; q < 2; ++q) landed(qfull + 8 * q, ((ph >> q) & 1) ^ 1);
        if (warp == 9) {
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            landed(drain, 0);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 9) tmem_free(tm, 512);
}

// One block per mask row: the 128-state tiles that keep a state, in order, their masks, and the kept states' number.
__global__ void __launch_bounds__(1024)
tdp_xattn_kept_kernel(const uint8_t *mask, int32_t S, int32_t *kept_n, int32_t *kept_states, int32_t *kept_tile, uint4 *kept_words,
                      uint4 *state_words)
{
    __shared__ uint32_t found[2][32];
    __shared__ int32_t states;
    const int32_t tiles = (S + kKeys - 1) / kKeys, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    const uint8_t *m = mask + row * S;
    const int32_t warps = blockDim.x >> 5;
    int32_t n = 0, mine = 0;
    if (threadIdx.x == 0) states = 0;
    for (int32_t t0 = 0, odd = 0; t0 < tiles; t0 += warps, odd ^= 1) {
        const int32_t t = t0 + warp;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t s = t * kKeys + 32 * i + lane;
            w[i] = __ballot_sync(~0u, t < tiles && s < S && m[s] != 0);
        }
        const bool any = (w[0] | w[1] | w[2] | w[3]) != 0;
        mine += __popc(w[0]) + __popc(w[1]) + __popc(w[2]) + __popc(w[3]);
        if (lane == 0 && t < tiles && state_words) state_words[row * tiles + t] = make_uint4(w[0], w[1], w[2], w[3]);
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
    __syncthreads();
    if (lane == 0) atomicAdd(&states, mine);        // whole numbers: their order is of no matter
    __syncthreads();
    if (threadIdx.x == 0) {
        kept_n[row] = n;
        kept_states[row] = states;
    }
}

}  // namespace tdp_xt
