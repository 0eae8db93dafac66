// tdp_xattn_grad_tc.cuh -- gradients of the bf16 cross attention on the tensor cores (tcgen05).
//
// Two kernels compute p = exp2(c s - lse) again.  The first walks the kept state tiles for each tile of
// 128 packed rows:   S = Q K^T, dP = dO V^T,  dS = p (dP - delta),  dQ += dS K,
// and writes delta = dO . O for the second, which walks the row tiles for each tile of 128 states:
//   S^T = K Q^T, dP^T = V dO^T,  dV += P^T dO,  dK += dS^T Q.
// Seven products where a single kernel would have five, but dK and dV then need no atomics and no
// exchange between blocks: a split over the rows writes fp32 parts that are joined in order.
// In both, scores and their gradients live in tensor memory; two warpgroups share the columns of a tile (each
// thread a lane and 64 columns) and write p and dS back as bf16 in place, as the next product's A operand (rounded by a
// relative 2^-8 at most, 0.0017 in the mean square, as the other operand and the gradient are):
//   warps 0-3, 4-7   columns 0-63, 64-127; the output
//   warp 8           loads tiles through tensor maps
//   warp 9           issues the products
//   warp 10          loads Q and dO (first kernel); each row's lse and delta (second)
//   warp 11          zeroes rows of a tile that must not count (their memory may hold anything, and 0 * NaN is not 0)
//
// 35840 rows, 16 heads of 128 on 4, 640 states: dq in 232 us (1.22 PFLOP/s, tensor pipe 51 % busy: one row tile, whose
// products wait for its softmax), dk and dv in 230 us (1.63 PFLOP/s, 69 %).  dP's columns are given back as soon as they
// are read: a tile of dq takes 1920 cycles for 2240 in one launch; both gradients at 16 heads of 64, 1000 states, 523 us for
// 544, at 128 columns 1 % less, the clock falling at the power limit.
#pragma once

#include "tdp_xattn_tc.cuh"

namespace tdp_xt {

template <int DP>
struct dq_smem {
    static constexpr int kTile = 128 * DP * 2;
    // A ring of O, then K and V in turn, of each item.  K stays from S to dQ: at five stages the next K and V still
    // come in time (with two K and two V stages S waited for its K in every round).
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr int kBytes = 1024 + (2 + kStages) * kTile + 512 + 1024;
};

template <int DP>
struct dkv_smem {
    static constexpr int kTile = 128 * DP * 2;
    static constexpr int kStages = DP == 128 ? 4 : 8;       // even: a stage always holds Q, or always dO
    static constexpr int kStats = 4;                        // row tiles of lse and delta
    static constexpr int kBytes = 1024 + (2 + kStages) * kTile + kStats * 1024 + 512;
};

// Rows whose mask keeps up to this many states in several state tiles: the first kernel walks the tiles twice.  Few states
// make delta as large as dP, and dO . O, with its O rounded to bf16, costs dS digits that delta = sum p dP over the row does
// not: a relative error of dQ of 0.0046 against 0.0023 at two states, 0.0032 at four, 0.0026 at 16, 0.00245 at 64 (scores of a
// spread of one; a softmax that a few of many states fill pays as much, whatever their number).  The first walk costs both
// gradients up to 1.7 times the time (35840 rows, 16 heads of 128, states in eight tiles: 2606 us against 1564): past 16
// states it gives less than a tenth of the error.  With one state tile the row's dP is all there and it is not needed.
constexpr int32_t kFewStates = 16;

// Item of the first kernel: a segment's tile of TT tokens, a head block, all kept state tiles.
__device__ __forceinline__ item dq_item_at(const tdp_geom &g, const xattn_args &a, int32_t w)
{
    item it;
    const int32_t blk = a.by_blocks.mod(w);
    it.head = a.by_heads.mod(w) * a.Gp;
    it.kvh = a.by_group.div(it.head);
    it.part = 0;
    it.seg = xattn_seg_fast(g, a, w);
    it.tok0 = (int64_t)blk * a.TT;
    it.left = (int32_t)(it.seg.T - it.tok0);
    const int32_t tiles = (a.S + kKeys - 1) / kKeys;
    it.keys.S = a.S;
    it.keys.tile = nullptr;
    it.keys.words = nullptr;
    it.keys.j0 = 0;
    it.keys.n = it.rounds = tiles;
    if (a.mask) {
        const int64_t m = a.per_tile ? (int64_t)it.seg.t * g.B + it.seg.b : it.seg.b;
        it.keys.n = a.kept_n[m];
        it.rounds = it.keys.n > 1 && a.kept_states[m] <= kFewStates ? 2 * it.keys.n : it.keys.n;
        it.keys.tile = a.kept_tile + m * tiles;
        it.keys.words = a.kept_words + m * tiles;
    }
    return it;
}

// log2 of the row's sum; a row with no sum gets +inf, which makes its probabilities zero.
__device__ __forceinline__ float row_lse2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
tdp_xattn_dq_kernel(const __grid_constant__ tdp_geom g, const __grid_constant__ xattn_args a,
                    const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_o,
                    const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, int32_t items)
{
    using SM = dq_smem<DP>;
    using T = __nv_bfloat16;
    constexpr int NST = SM::kStages;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t q_s = base, do_s = q_s + SM::kTile, kv_s = do_s + SM::kTile, bars = kv_s + NST * SM::kTile, stat_s = bars + 512;
    const uint32_t full = bars, empty = full + 8 * NST, clean = empty + 8 * NST, rfull = clean + 32, rempty = rfull + 16,
                   sfull = rempty + 16, pfull = sfull + 16, dsfull = pfull + 8,
                   done = dsfull + 8, drain = done + 8, pread = drain + 8;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead_flag;
    volatile int *dead = &dead_flag;
    const int32_t warp = role(), lane = threadIdx.x & 31;
    if (warp == 9) tmem_alloc(smem_u32(&tmem_slot), 512);
    if (threadIdx.x == 0) {
        dead_flag = 0;
        // a tile is given back by its last reader and, where there is a mask, by the cleaning warp, which waits for every
        // tile: a stage filled again before it has looked would put its wait a phase behind
        for (int i = 0; i < NST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, a.mask ? 2 : 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(clean + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(rfull + 8 * i, 1);            // Q, dO
            mbar_init(rempty + 8 * i, i ? 2 : 1);   // dO is given back by the products and by delta
            mbar_init(sfull + 8 * i, 1);
        }
        mbar_init(pfull, 1);
        mbar_init(pread, 8);
        mbar_init(dsfull, 8);
        mbar_init(done, 1);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = tmem_slot;              // S: columns 0-127 and 128-255, taking turns; dP 256-383; dQ 384-
    tdp_pdl_trigger();
    tdp_pdl_wait();

    bool ok = true;
    ring<NST> kv = {0, 0};
    uint32_t n_done = 0, n_items = 0;           // state tiles and items so far
    if (warp < 8) {
        regs_inc<216>();
        const int32_t half = warp >> 2, r = threadIdx.x & 127, rt = r / a.Gp, rh = r - rt * a.Gp;
        const uint32_t lanes = tm + ((uint32_t)(warp & 3) << 21);
        const float c = a.scale * kLog2e;
        const bool wide = a.D % 16 == 0 && (reinterpret_cast<uintptr_t>(a.dq) & 31) == 0;      // whole sectors
        // A row's sum of its two threads' parts, in one order.
        auto both = [&](float x) {
            float other;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(stat_s + 512 * half + 4 * r), "f"(x) : "memory");
            asm volatile("bar.sync 1, 256;" ::: "memory");
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(stat_s + 512 * (half ^ 1) + 4 * r) : "memory");
            asm volatile("bar.sync 1, 256;" ::: "memory");
            return half ? other + x : x + other;
        };
        // After a lost wait, another thread's too, delta and dQ are NaN: a row's sums have parts of several threads, and the
        // kernel that follows must not take a delta of what was not there.
        auto sound = [&] { return ok && !*dead; };
        // An item's lse and delta = dO . O, made while the products of the item before run out: each thread half of a
        // row's products, the halves joined through shared memory.
        item it;
        float l, d;
        auto ahead = [&](int32_t w) {
            it.left = 0;
            if (w >= items) return;
            it = dq_item_at(g, a, w);
            if (it.left <= 0 || it.keys.n == 0) return;
            const bool mine = rt < a.TT && rt < it.left;
            const int32_t h = ((int32_t)(it.seg.row0 + it.tok0) + rt) * a.Hq + it.head + rh;
            l = -row_lse2(mine ? a.lse[h] : -INFINITY);
            ok = ok && mbar_wait(full + 8 * kv.st, kv.ph, dead) && mbar_wait(rfull + 8, n_items & 1, dead);
            ++n_items;
            float sum = 0.f;
            const uint32_t o_t = kv_s + kv.st * SM::kTile;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                const int32_t col = half * (DP / 16) + i;       // 16-byte chunk
                const uint32_t off = (col / 8) * 16384 + panel_off(r, col & 7);
                uint4 x, y;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(o_t + off) : "memory");
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(do_s + off) : "memory");
                float fx[8], fy[8];
                tdp_elem<1>::unpack(x, fx);
                tdp_elem<1>::unpack(y, fy);
#pragma unroll
                for (int u = 0; u < 8; ++u) sum = fmaf(fx[u], fy[u], sum);
            }
            d = both(sum);
            if (warp == 0 && lane == 0) {
                mbar_arrive(empty + 8 * kv.st);
                mbar_arrive(rempty + 8);
            }
            if (mine && half == 0) a.delta[h] = sound() ? d : NAN;
            d = -d;
            const uint32_t to = kv.st + 1 + 2 * it.rounds, rounds = to / NST;
            kv.st = to - rounds * NST;
            kv.ph ^= rounds & 1;
        };
        ahead(blockIdx.x);
        for (int32_t w = blockIdx.x; w < items; w += gridDim.x) {
            const int32_t n = it.keys.n;
            if (it.left <= 0) {
                ahead(w + gridDim.x);
                continue;
            }
            const bool mine = rt < a.TT && rt < it.left;
            const int32_t h = ((int32_t)(it.seg.row0 + it.tok0) + rt) * a.Hq + it.head + rh;
            if (n > 0) {
                // delta from the probabilities: of the only tile, or of all tiles in a first walk, whose dS is zero
                const int32_t rounds = it.rounds, first = rounds - n;
                const bool tally = n == 1 || first > 0;
                float sum = 0.f;
                const uint32_t done_ph = (n_items & 1) ^ 1;
                const uint64_t c2 = pair(c, c), l2 = pair(l, l);
                uint64_t d2 = pair(d, d);
#pragma unroll 1
                for (int32_t j = 0; j < rounds && (ok || tally); ++j) {     // tally: all threads meet in both()
                    const uint32_t buf = n_done & 1, S = lanes + 128 * buf + 64 * half, P = lanes + 256 + 64 * half;
                    const uint4 mk = it.keys.mask(j < first ? j : j - first);
                    ok = ok && mbar_wait(sfull + 8 * buf, (n_done >> 1) & 1, dead) && mbar_wait(pfull, n_done & 1, dead);
                    ++n_done;
                    fence_after();
                    uint32_t s[64], e[64];
                    tmem_ld32(S, s);
                    tmem_ld32(S + 32, s + 32);
                    tmem_ld32(P, e);
                    tmem_ld32(P + 32, e + 32);
                    tmem_wait_ld();
                    tmem_have32(s);
                    tmem_have32(s + 32);
                    tmem_have32(e);
                    tmem_have32(e + 32);
                    // dP may be made anew: the next tile's runs under this one's arithmetic
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pread);
#pragma unroll
                    for (int u = 0; u < 32; ++u) {
                        float x, y;
                        unpair(fma2(pair(__uint_as_float(s[2 * u]), __uint_as_float(s[2 * u + 1])), c2, l2), x, y);
                        s[2 * u] = __float_as_uint(exp2_fast(x));
                        s[2 * u + 1] = __float_as_uint(exp2_fast(y));
                    }
                    uint32_t w0 = half ? mk.z : mk.x, w1 = half ? mk.w : mk.y;
                    if (n == 1 || j < first) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            if ((w0 >> u) & 1) sum = fmaf(__uint_as_float(s[u]), __uint_as_float(e[u]), sum);
                            if ((w1 >> u) & 1) sum = fmaf(__uint_as_float(s[32 + u]), __uint_as_float(e[32 + u]), sum);
                        }
                        if (j + 1 >= first) {
                            sum = both(sum);
                            if (mine && half == 0) a.delta[h] = sound() ? sum : NAN;
                            d2 = pair(-sum, -sum);
                        }
                        if (j < first) w0 = w1 = 0;
                    }
#pragma unroll
                    for (int u = 0; u < 32; ++u) {
                        float x, y;
                        unpair(mul2(pair(__uint_as_float(s[2 * u]), __uint_as_float(s[2 * u + 1])),
                                    add2(pair(__uint_as_float(e[2 * u]), __uint_as_float(e[2 * u + 1])), d2)), x, y);
                        s[2 * u] = __float_as_uint(x);
                        s[2 * u + 1] = __float_as_uint(y);
                    }
                    if ((w0 & w1) != ~0u) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            if (!((w0 >> u) & 1)) s[u] = 0;
                            if (!((w1 >> u) & 1)) s[32 + u] = 0;
                        }
                    }
                    // dS as bf16 over this half's scores
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t b[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            b[u] = tdp_pack_bf16x2(__uint_as_float(s[32 * v + 2 * u]), __uint_as_float(s[32 * v + 2 * u + 1]));
                        tmem_st16(S + 16 * v, b);
                    }
                    tmem_wait_st();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(dsfull);
                }
                ahead(w + gridDim.x);
                if (ok) ok = mbar_wait(done, done_ph, dead);
                fence_after();
            } else {
                if (mine && half == 0) a.delta[h] = 0.f;
                ahead(w + gridDim.x);
            }
            // dQ, half of the columns each; a lost wait leaves NaN
            T *dst = static_cast<T *>(a.dq) + (int64_t)h * a.D;
            const float f = sound() ? a.scale : NAN;
#pragma unroll 1
            for (int i = half * (DP / 64); i < (half + 1) * (DP / 64); ++i) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(lanes + 384 + 32 * i, o);
                    tmem_wait_ld();
                    tmem_have32(o);
                } else {
#pragma unroll
                    for (int u = 0; u < 32; ++u) o[u] = 0;
                }
                uint32_t b[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) b[u] = tdp_pack_bf16x2(__uint_as_float(o[2 * u]) * f, __uint_as_float(o[2 * u + 1]) * f);
                if (mine) {
                    if (wide) {
#pragma unroll
                        for (int u = 0; u < 16; u += 8)
                            if (32 * i + 2 * u < a.D) st_global32(dst + 32 * i + 2 * u, b + u);
                    } else {
#pragma unroll
                        for (int u = 0; u < 16; u += 4)
                            if (32 * i + 2 * u < a.D) *reinterpret_cast<uint4 *>(dst + 32 * i + 2 * u) = make_uint4(b[u], b[u + 1], b[u + 2], b[u + 3]);
                    }
                }
                __syncwarp();
            }
            fence_before();
        }
    } else {
        regs_dec<72>();
        uint32_t kc = 0;                        // K tiles so far
        for (int32_t w = blockIdx.x; w < items; w += gridDim.x) {
            const item it = dq_item_at(g, a, w);
            const int32_t tiles = it.keys.n, n = it.rounds;     // state tiles; those of all walks
            if (it.left <= 0 || n == 0 || !ok) continue;
            const int32_t row = (int32_t)(it.seg.row0 + it.tok0);
            const uint32_t ph = n_items & 1;
            const uint32_t row_bytes = (uint32_t)(a.Gp * a.TT) * DP * 2;
            if (warp == 8) {
                // O, K 0, V 0, K 1, ...
#pragma unroll 1
                for (int32_t i = -1; i < 2 * n; ++i) {
                    const bool v = i & 1;
                    const int32_t head = (v ? a.v_head : a.k_head) > 0 ? it.kvh : 0, b = (v ? a.v_item : a.k_item) > 0 ? it.seg.b : 0;
                    const int32_t state = i < 0 ? 0 : it.keys.at((i >> 1) < tiles ? i >> 1 : (i >> 1) - tiles) * kKeys;
                    if (!(ok = mbar_wait(empty + 8 * kv.st, kv.ph ^ 1, dead))) break;
                    if (elect_one()) {
                        const uint32_t dst = kv_s + kv.st * SM::kTile, bar = full + 8 * kv.st;
                        mbar_expect(bar, i < 0 ? row_bytes : (uint32_t)SM::kTile);
                        for (int p = 0; p < DP / 64; ++p) {
                            if (i < 0) tma_load3(dst + p * 16384, &map_o, bar, 64 * p, it.head, row);
                            else tma_load4(dst + p * 16384, v ? &map_v : &map_k, bar, 64 * p, head, state, b);
                        }
                    }
                    __syncwarp();
                    kv.next();
                }
            } else if (warp == 10) {
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    if (!(ok = mbar_wait(rempty + 8 * i, ph ^ 1, dead))) break;
                    if (elect_one()) {
                        mbar_expect(rfull + 8 * i, row_bytes);
                        for (int p = 0; p < DP / 64; ++p)
                            tma_load3(base + i * SM::kTile + p * 16384, i ? &map_do : &map_q, rfull + 8 * i, 64 * p, it.head, row);
                    }
                    __syncwarp();
                }
            } else if (warp == 9) {
                constexpr uint32_t id_s = idesc(128, 128, false, false), id_q = idesc(128, DP, false, true);
                const uint32_t q_d = desc_rows(q_s), do_d = desc_rows(do_s);
                // A product of eight (DP / 16) steps.  The tensor cores queue two of them, some 128 cycles, and a wait
                // takes longer: the next product's barrier is looked at before the last two steps are issued.
                bool there = false;
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    if (!there) ok = ok && mbar_wait(bar, parity, dead);
                    there = false;
                    __syncwarp();
                    return ok;
                };
                auto rows = [&](uint32_t d, uint32_t x, uint32_t y, uint32_t end, uint32_t end2, uint32_t end3, uint32_t next, uint32_t parity) {
                    auto step = [&](int i) {
                        const uint32_t o = (i / 4) * (16384 >> 4) + (i % 4) * 2;
                        mma_ss(d, x + o, y + o, id_s, i > 0);
                    };
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < DP / 16 - 2; ++i) step(i);
                    }
                    there = next && mbar_test(next, parity);
                    __syncwarp();
                    if (elect_one()) {
                        step(DP / 16 - 2);
                        step(DP / 16 - 1);
                        mma_commit(end);
                        if (end2) mma_commit(end2);
                        if (end3) mma_commit(end3);
                    }
                    __syncwarp();
                };
                kv.next();                      // O
                uint32_t k_prev = 0;
                // round j: S of state tile j + 1 ahead, dP of j + 1 once that of j has been read, dQ of j once dS of j is there
#pragma unroll 1
                for (int32_t j = -1; j < n; ++j) {
                    const uint32_t b1 = n_done & 1, k1 = kv.st;     // n_done: S products so far
                    if (j + 1 < n) {
                        if (j < 0 && !(ok = mbar_wait(rfull, ph, dead))) break;
                        // K comes by way of the cleaning warp where there is a mask
                        if (!(a.mask ? wait(clean + 8 * (kc & 3), (kc >> 2) & 1) : wait(full + 8 * k1, kv.ph))) break;
                        ++kc;
                        rows(tm + 128 * b1, q_d, desc_rows(kv_s + k1 * SM::kTile), sfull + 8 * b1, j + 2 == n ? rempty : 0, 0,
                             j >= 0 ? pread : 0, (n_done - 1) & 1);
                        ++n_done;
                        kv.next();
                    }
                    const uint32_t tile = (j + 1 < n ? n_done : n_done + 1) & 1;         // parity of tile j
                    if (j + 1 < n) {
                        if (j < 0 && !(ok = mbar_wait(rfull + 8, ph, dead))) break;
                        if (j >= 0) {
                            if (!wait(pread, tile)) break;
                            fence_after();
                        }
                        if (!wait(full + 8 * kv.st, kv.ph)) break;
                        rows(tm + 256, do_d, desc_rows(kv_s + kv.st * SM::kTile), pfull, empty + 8 * kv.st, j + 2 == n ? rempty + 8 : 0,
                             j >= 0 ? dsfull : 0, tile);
                        kv.next();
                    }
                    if (j >= 0) {
                        if (!wait(dsfull, tile)) break;
                        fence_after();
                    }
                    if (j >= 0) {
                        const uint32_t ds = tm + 128 * tile, y0 = desc_cols(kv_s + k_prev * SM::kTile, 16384);
                        auto step = [&](int i) { mma_ts(tm + 384, ds + 64 * (i / 4) + 8 * (i % 4), y0 + i * (2048 >> 4), id_q, j > 0 || i > 0); };
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 6; ++i) step(i);
                        }
                        there = j + 2 < n && (a.mask ? mbar_test(clean + 8 * (kc & 3), (kc >> 2) & 1) : mbar_test(full + 8 * kv.st, kv.ph));
                        __syncwarp();
                        if (elect_one()) {
                            step(6);
                            step(7);
                            mma_commit(empty + 8 * k_prev);
                            if (j + 1 == n) mma_commit(done);
                        }
                        __syncwarp();
                    }
                    k_prev = k1;
                }
            } else if (a.mask) {
                // O, then K and V of each state tile: every one is waited for, in order, and given back
#pragma unroll 1
                for (int32_t i = -1; i < 2 * n; ++i) {
                    if (!(ok = mbar_wait(full + 8 * kv.st, kv.ph, dead))) break;
                    const bool k = i >= 0 && !(i & 1);
                    if (k) {
                        zero_dropped<DP>(kv_s + kv.st * SM::kTile, it.keys.mask((i >> 1) < tiles ? i >> 1 : (i >> 1) - tiles), lane);
                        fence_async();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (k) mbar_arrive(clean + 8 * (kc & 3));
                        mbar_arrive(empty + 8 * kv.st);
                    }
                    kc += k;
                    kv.next();
                }
            }
            ++n_items;
        }
    }
    // nothing may land, or be on its way, after the block has gone
    auto landed = [&](uint32_t bar, uint32_t parity) {
#pragma unroll 1
        for (uint32_t i = 0; i < kWaitRounds && !mbar_try(bar, parity); ++i) {
        }
    };
    if (warp == 8) {
        for (uint32_t i = 0; i < NST; ++i) landed(full + 8 * i, i < kv.st ? kv.ph : kv.ph ^ 1);
    } else if (warp == 10) {
        for (int i = 0; i < 2; ++i) landed(rfull + 8 * i, (n_items & 1) ^ 1);
    } else if (warp == 9) {
        if (elect_one()) mma_commit(drain);
        __syncwarp();
        landed(drain, 0);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 9) tmem_free(tm, 512);
}

// Walk over the row tiles of one batch item that meet a tile of states: the part's units [u, last), unit u = block
// u % blocks of the item's segment u / blocks; a segment's run of blocks at a time.
struct row_walk {
    int32_t u, last;
    tdp_seg seg;
    int32_t blk, end;               // the run's blocks
    uint4 words;                    // kept states of the tile
    __device__ __forceinline__ bool next(const tdp_geom &g, const xattn_args &a, int32_t b, int32_t tile)
    {
        while (u < last) {
            const int32_t sg = a.by_blocks.div(u);
            seg = xattn_seg_fast(g, a, sg * g.B + b);
            blk = u - sg * a.blocks;
            end = min(blk + last - u, (int32_t)((seg.T + a.TT - 1) / a.TT));
            u = (sg + 1) * a.blocks;
            if (a.mask) {
                const int64_t m = a.per_tile ? (int64_t)seg.t * g.B + seg.b : seg.b;
                words = a.state_words[m * ((a.S + kKeys - 1) / kKeys) + tile];
            } else {
                key_list k;
                k.tile = nullptr;
                k.words = nullptr;
                k.j0 = tile;
                k.S = a.S;
                words = k.mask(0);
            }
            if (blk < end && (words.x | words.y | words.z | words.w) != 0) return true;
        }
        return false;
    }
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
tdp_xattn_dkv_kernel(const __grid_constant__ tdp_geom g, const __grid_constant__ xattn_args a,
                     const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
                     const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using SM = dkv_smem<DP>;
    using T = __nv_bfloat16;
    constexpr int NST = SM::kStages, NSS = SM::kStats;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t k_s = base, v_s = k_s + SM::kTile, r_s = v_s + SM::kTile, stat_s = r_s + NST * SM::kTile, bars = stat_s + NSS * 1024;
    const uint32_t full = bars, empty = full + 8 * NST, clean = empty + 8 * NST, tfull = clean + 8 * NST, tempty = tfull + 8 * NSS,
                   kvfull = tempty + 8 * NSS, sfull = kvfull + 8, dpfull = sfull + 8, pready = dpfull + 8, dsready = pready + 8,
                   drain = dsready + 8;
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
        for (int i = 0; i < NSS; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 8);
        }
        mbar_init(kvfull, 1);
        mbar_init(sfull, 1);
        mbar_init(dpfull, 1);
        mbar_init(pready, 8);
        mbar_init(dsready, 8);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // rows of a tile past Gp * TT are never loaded: zero once
    for (uint32_t i = threadIdx.x; i < NST * SM::kTile / 16; i += kThreads) st_zero16(r_s + 16 * i);
    fence_async();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = tmem_slot;              // S^T 0-127, dP^T 128-255, dV 256-, dK 384-
    tdp_pdl_trigger();
    tdp_pdl_wait();

    const int32_t tiles = (a.S + kKeys - 1) / kKeys;
    int32_t w = blockIdx.x;
    const int32_t tile = w % tiles;
    w /= tiles;
    const int32_t kvh = w % a.Hkv;
    w /= a.Hkv;
    const int32_t part = w % a.split, b = w / a.split;
    const int32_t units = (a.flat ? 1 : g.nt) * a.blocks, hbs = a.G / a.Gp;     // head blocks that share the key head
    row_walk wk;
    wk.u = min(units, part * a.part);
    wk.last = min(units, wk.u + a.part);

    // every role walks the same row tiles, each for the head blocks in turn
    bool ok = true, any = false;
    uint32_t n = 0;                             // row tiles so far
    if (warp < 8) {
        regs_inc<216>();
        const int32_t half = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = tm + ((uint32_t)(warp & 3) << 21), S = lanes + 64 * half, P = lanes + 128 + 64 * half;
        const float c = a.scale * kLog2e;
        const uint64_t c2 = pair(c, c);
        while (ok && wk.next(g, a, b, tile)) {
            const uint32_t word = r < 64 ? (r < 32 ? wk.words.x : wk.words.y) : (r < 96 ? wk.words.z : wk.words.w);
            const bool kept = (word >> lane) & 1;
            const int32_t tiles_in = (wk.end - wk.blk) * hbs;
#pragma unroll 1
            for (int32_t i = 0; i < tiles_in && ok; ++i, ++n) {
                const uint32_t ss = n % NSS, st = stat_s + ss * 1024 + 256 * half;
                any = true;
                ok = mbar_wait(tfull + 8 * ss, (n / NSS) & 1, dead) && mbar_wait(sfull, n & 1, dead);
                fence_after();
                uint32_t s[64], x32[32];
                tmem_ld32(S, s);
                tmem_ld32(S + 32, s + 32);
                tmem_wait_ld();
                tmem_have32(s);
                tmem_have32(s + 32);
                // p, kept in registers for dS; as bf16 over this half's scores
#pragma unroll
                for (int v = 0; v < 2; ++v) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        uint64_t l0, l1;
                        float p0, p1, p2, p3;
                        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(l0), "=l"(l1) : "r"(st + 128 * v + 16 * u));
                        uint32_t *q = s + 32 * v + 4 * u;
                        unpair(fma2(pair(__uint_as_float(q[0]), __uint_as_float(q[1])), c2, l0), p0, p1);
                        unpair(fma2(pair(__uint_as_float(q[2]), __uint_as_float(q[3])), c2, l1), p2, p3);
                        p0 = kept ? exp2_fast(p0) : 0.f;
                        p1 = kept ? exp2_fast(p1) : 0.f;
                        p2 = kept ? exp2_fast(p2) : 0.f;
                        p3 = kept ? exp2_fast(p3) : 0.f;
                        q[0] = __float_as_uint(p0);
                        q[1] = __float_as_uint(p1);
                        q[2] = __float_as_uint(p2);
                        q[3] = __float_as_uint(p3);
                        x32[2 * u] = tdp_pack_bf16x2(p0, p1);
                        x32[2 * u + 1] = tdp_pack_bf16x2(p2, p3);
                    }
                    tmem_st16(S + 16 * v, x32);
                }
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready);
                ok = ok && mbar_wait(dpfull, n & 1, dead);
                fence_after();
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    uint32_t b16[16];
                    tmem_ld32(P + 32 * v, x32);
                    tmem_wait_ld();
                    tmem_have32(x32);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        uint64_t d0, d1;
                        float y0, y1, y2, y3;
                        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(d0), "=l"(d1) : "r"(st + 512 + 128 * v + 16 * u));
                        const uint32_t *q = s + 32 * v + 4 * u, *d = x32 + 4 * u;
                        unpair(mul2(pair(__uint_as_float(q[0]), __uint_as_float(q[1])), add2(pair(__uint_as_float(d[0]), __uint_as_float(d[1])), d0)), y0, y1);
                        unpair(mul2(pair(__uint_as_float(q[2]), __uint_as_float(q[3])), add2(pair(__uint_as_float(d[2]), __uint_as_float(d[3])), d1)), y2, y3);
                        b16[2 * u] = kept ? tdp_pack_bf16x2(y0, y1) : 0u;      // a dropped state's dP may be NaN
                        b16[2 * u + 1] = kept ? tdp_pack_bf16x2(y2, y3) : 0u;
                    }
                    tmem_st16(P + 16 * v, b16);
                }
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(dsready);
                    mbar_arrive(tempty + 8 * ss);
                }
            }
        }
        if (ok) ok = mbar_wait(drain, 0, dead);
        fence_after();
        // first warpgroup dV, second dK
        const int32_t state = tile * kKeys + r;
        const int64_t at = (((int64_t)b * a.S + state) * a.Hkv + kvh) * a.D;
        // a wait that any thread of the block has lost leaves NaN: the columns of a tile are shared
        const float f = !ok || *dead ? NAN : half ? a.scale : 1.f;
        float *pf = (half ? a.pk : a.pv) + (int64_t)part * g.B * a.S * a.Hkv * a.D + at;
        T *pb = static_cast<T *>(half ? a.dk : a.dv) + at;
#pragma unroll 1
        for (int i = 0; i < DP / 32; ++i) {
            uint32_t o[32];
            if (any) {
                tmem_ld32(lanes + 256 + 128 * half + 32 * i, o);
                tmem_wait_ld();
                tmem_have32(o);
            } else {
#pragma unroll
                for (int u = 0; u < 32; ++u) o[u] = 0;
            }
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
            if (state < a.S) {
#pragma unroll
                for (int u = 0; u < 32; u += 8) {
                    if (32 * i + u >= a.D) continue;
                    if (a.split > 1) {
                        st_global32(pf + 32 * i + u, o + u);
                    } else {
                        float y[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) y[x] = __uint_as_float(o[u + x]);
                        *reinterpret_cast<uint4 *>(pb + 32 * i + u) = tdp_elem<1>::pack(y);
                    }
                }
            }
            __syncwarp();
        }
        fence_before();
    } else {
        regs_dec<72>();
        uint32_t ti = 0;                        // Q and dO tiles so far
        constexpr uint32_t id_s = idesc(128, 128, false, false), id_o = idesc(128, DP, false, true);
        // A product of eight (DP / 16) steps.  The tensor cores queue two of them, some 128 cycles, and a wait with what
        // surrounds it takes longer: the next product's barrier is looked at before the last two steps are issued.
        bool there = false;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (!there) ok = ok && mbar_wait(bar, parity, dead);
            __syncwarp();
            return ok;
        };
        // both operands row-major over the head dimension
        auto rows = [&](uint32_t d, uint32_t x, uint32_t y, uint32_t done, uint32_t next, uint32_t parity) {
            auto step = [&](int i) {
                const uint32_t o = (i / 4) * (16384 >> 4) + (i % 4) * 2;       // next panel, or 32 bytes
                mma_ss(d, x + o, y + o, id_s, i > 0);
            };
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < DP / 16 - 2; ++i) step(i);
            }
            there = mbar_test(next, parity);
            __syncwarp();
            if (elect_one()) {
                step(DP / 16 - 2);
                step(DP / 16 - 1);
                mma_commit(done);
            }
            __syncwarp();
        };
        // A from tensor memory, 64 columns of it at each half; B: a row tile read by columns
        auto cols = [&](uint32_t d, uint32_t p, uint32_t y, bool acc, uint32_t done, uint32_t next, uint32_t parity) {
            auto step = [&](int i) { mma_ts(d, p + 64 * (i / 4) + 8 * (i % 4), y + i * (2048 >> 4), id_o, acc || i > 0); };
            fence_after();
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 6; ++i) step(i);
            }
            there = next && mbar_test(next, parity);
            __syncwarp();
            if (elect_one()) {
                step(6);
                step(7);
                mma_commit(done);
            }
            __syncwarp();
        };
        if (warp == 8 && elect_one()) {
            const int32_t kh = a.k_head > 0 ? kvh : 0, kb = a.k_item > 0 ? b : 0, vh = a.v_head > 0 ? kvh : 0, vb = a.v_item > 0 ? b : 0;
            mbar_expect(kvfull, 2 * SM::kTile);
            for (int p = 0; p < DP / 64; ++p) {
                tma_load4(k_s + p * 16384, &map_k, kvfull, 64 * p, kh, tile * kKeys, kb);
                tma_load4(v_s + p * 16384, &map_v, kvfull, 64 * p, vh, tile * kKeys, vb);
            }
        }
        __syncwarp();
        if (warp == 9) ok = mbar_wait(kvfull, 0, dead);
        // warp 10: token in the tile, and place from the tile's first row, of the lane's four rows
        int32_t st_tok[4], st_at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t x = 32 * i + lane, rt = x / a.Gp;
            st_tok[i] = rt < a.TT ? rt : INT32_MAX;
            st_at[i] = rt * a.Hq + x - rt * a.Gp;
        }
        // warp 9 runs one tile behind itself: dK and dP of a tile come after S of the next
        uint32_t q_prev = 0;
        while (ok && wk.next(g, a, b, tile)) {
            int32_t hb = 0, tok = wk.blk * a.TT;        // head block and first token of the tile in its segment
            const int32_t tiles_in = (wk.end - wk.blk) * hbs;
#pragma unroll 1
            for (int32_t t = 0; t < tiles_in && ok; ++t, ++n) {
                const int32_t head = kvh * a.G + hb * a.Gp, row = (int32_t)wk.seg.row0 + tok, left = (int32_t)wk.seg.T - tok;
                if (++hb == hbs) {
                    hb = 0;
                    tok += a.TT;
                }
                if (warp == 8) {
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t st = ti % NST;
                        if (!(ok = mbar_wait(empty + 8 * st, ((ti / NST) & 1) ^ 1, dead))) break;
                        ++ti;
                        if (elect_one()) {
                            mbar_expect(full + 8 * st, (uint32_t)(a.Gp * a.TT) * DP * 2);
                            for (int p = 0; p < DP / 64; ++p)
                                tma_load3(r_s + st * SM::kTile + p * 16384, i ? &map_do : &map_q, full + 8 * st, 64 * p, head, row);
                        }
                        __syncwarp();
                    }
                } else if (warp == 9) {
                    const uint32_t qs = ti % NST, ds = qs + 1, tph = (ti / NST) & 1;
                    const uint32_t q_t = desc_rows(r_s + qs * SM::kTile), do_t = desc_rows(r_s + ds * SM::kTile);
                    const uint32_t q_p = desc_cols(r_s + q_prev * SM::kTile, 16384), do_p = desc_cols(r_s + (q_prev + 1) * SM::kTile, 16384);
                    ti += 2;
                    if (n > 0) {
                        // dV of the tile before, whose probabilities lie in S
                        if (!wait(pready, (n - 1) & 1)) break;
                        cols(tm + 256, tm, do_p, n > 1, empty + 8 * (q_prev + 1), clean + 8 * qs, tph);
                    }
                    if (!wait(clean + 8 * qs, tph)) break;
                    rows(tm, desc_rows(k_s), q_t, sfull, n > 0 ? dsready : clean + 8 * ds, n > 0 ? (n - 1) & 1 : tph);
                    if (n > 0) {
                        // dK of the tile before, whose dS lies in dP
                        if (!wait(dsready, (n - 1) & 1)) break;
                        cols(tm + 384, tm + 128, q_p, n > 1, empty + 8 * q_prev, clean + 8 * ds, tph);
                    }
                    if (!wait(clean + 8 * ds, tph)) break;
                    rows(tm + 128, desc_rows(v_s), do_t, dpfull, pready, n & 1);
                    q_prev = qs;
                } else if (warp == 10) {
                    const uint32_t ss = n % NSS, dst = stat_s + ss * 1024;
                    if (!(ok = mbar_wait(tempty + 8 * ss, ((n / NSS) & 1) ^ 1, dead))) break;
                    // all eight loads at once, from the tile's first row for rows that are not there: behind a condition each
                    // they came one after the other, 6000 cycles a tile where the products take 2000
                    const int32_t h0 = row * a.Hq + head;
                    float l[4], d[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t h = h0 + (st_tok[i] < left ? st_at[i] : 0);
                        l[i] = a.lse[h];
                        d[i] = __ldcg(a.delta + h);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool on = st_tok[i] < left;
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + 4 * (32 * i + lane)), "f"(on ? -row_lse2(l[i]) : -INFINITY) : "memory");
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + 512 + 4 * (32 * i + lane)), "f"(on ? -d[i] : 0.f) : "memory");
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tfull + 8 * ss);
                } else {
                    // rows past the segment's end belong to another tile
                    const int32_t rows_in = min(left, a.TT) * a.Gp, rows_all = a.TT * a.Gp;
                    constexpr int C = DP / 8;
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t st = ti % NST;
                        if (!(ok = mbar_wait(full + 8 * st, (ti / NST) & 1, dead))) break;
                        ++ti;
#pragma unroll 1
                        for (int32_t x = rows_in * C + lane; x < rows_all * C; x += 32)
                            st_zero16(r_s + st * SM::kTile + (x % C / 8) * 16384 + panel_off(x / C, x % C & 7));
                        fence_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(clean + 8 * st);
                    }
                }
            }
        }
        auto landed = [&](uint32_t bar, uint32_t parity) {
#pragma unroll 1
            for (uint32_t i = 0; i < kWaitRounds && !mbar_try(bar, parity); ++i) {
            }
        };
        if (warp == 9) {
            if (n > 0 && ok) {
                if (wait(pready, (n - 1) & 1))
                    cols(tm + 256, tm, desc_cols(r_s + (q_prev + 1) * SM::kTile, 16384), n > 1, empty + 8 * (q_prev + 1), dsready, (n - 1) & 1);
                if (wait(dsready, (n - 1) & 1))
                    cols(tm + 384, tm + 128, desc_cols(r_s + q_prev * SM::kTile, 16384), n > 1, empty + 8 * q_prev, 0, 0);
            }
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            landed(drain, 0);
        } else if (warp == 8) {
            landed(kvfull, 0);
            for (uint32_t i = ti > NST ? ti - NST : 0; i < ti; ++i) landed(full + 8 * (i % NST), (i / NST) & 1);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 9) tmem_free(tm, 512);
}

}  // namespace tdp_xt
