// tdp_rope.cu -- rotary positions: every head of a tile-major row turned by the row's position, and back.
//
// Pair i of a head, (a, b), belongs to an axis and has a frequency f_i: with p the row's position on that axis,
//   a' = scale (a cos(p f) - b sin(p f)),  b' = scale (a sin(p f) + b cos(p f));  the gradient turns by -p f.
// An angle is kept in turns: p f / 2 pi, of which only the fraction counts, is the low 64 bits of the product of an integer
// position and the frequency in 2^-64 turns.  No reduction loses digits however far the position is: 2^32 positions off
// the origin this is 2^-30 turns off, what fp32 then holds of it 2^-28 (2^-24 in bf16's fast form), and 64-bit floats, a fiftieth of the rate of 32-bit ones here, are not needed.
//
// Bound by memory.  A thread makes the sines of its pairs once and takes them through the heads of its row, 16 bytes at
// a time where the layout allows, several heads' loads ahead.
#include <algorithm>
#include <cmath>

#include "tdp.h"
#include "tdp_internal.h"
#include "tdp_rows.cuh"
#include "tdp_tc.cuh"

namespace {

using tdp_tc::fma2;
using tdp_tc::mul2;
using tdp_tc::pair;
using tdp_tc::unpair;

constexpr int kRopeThreads = 256;
constexpr int kRopeAhead = 4;               // heads whose loads a thread has under way
constexpr double kInvFourPiHi = 0.07957747154594767;        // 1 / (4 pi), and what it lacks
constexpr double kInvFourPiLo = -4.9196691687956215e-18;

struct rope_args {
    const void *x;
    const int32_t *pos;
    const int64_t *table;
    void *out;
    int64_t x_row, x_head, out_row, out_head;       // strides in bytes
    int32_t heads, pairs;
    int32_t turned, items;      // items of a head: those of pairs, and with them those behind the pairs
    int32_t groups;             // heads side by side
    int32_t rows;               // rows of a block
    int32_t blocks;             // blocks of the largest segment
    int32_t middle;
    float sign, scale;
    fast_div by_blocks, by_team, by_items, by_B, by_nH, by_nW;
};

// W elements as fp32.
template <int BF16, int W>
__device__ __forceinline__ void load(const unsigned char *p, uint32_t *u)
{
    constexpr int B = W * (BF16 ? 2 : 4);
    if (B == 16) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
        u[0] = v.x;
        u[1] = v.y;
        u[2] = v.z;
        u[3] = v.w;
    } else if (B == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
        u[0] = v.x;
        u[1] = v.y;
    } else if (B == 4) {
        u[0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
    } else {
        u[0] = __ldcs(reinterpret_cast<const unsigned short *>(p));
    }
}
template <int BF16, int W>
__device__ __forceinline__ void store(unsigned char *p, const uint32_t *u)
{
    constexpr int B = W * (BF16 ? 2 : 4);
    if (B == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    else if (B == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(u[0], u[1]);
    else if (B == 4) *reinterpret_cast<uint32_t *>(p) = u[0];
    else *reinterpret_cast<unsigned short *>(p) = (unsigned short)u[0];
}
template <int BF16, int W>
__device__ __forceinline__ void unpack(const uint32_t *u, float *f)
{
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = BF16 ? (i & 1 ? tdp_bf16_hi(u[i / 2]) : tdp_bf16_lo(u[i / 2])) : __uint_as_float(u[i]);
}
template <int BF16, int W>
__device__ __forceinline__ void pack(const float *f, uint32_t *u)
{
    if (!BF16) {
#pragma unroll
        for (int i = 0; i < W; ++i) u[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 2) u[i / 2] = tdp_pack_bf16x2(f[i], i + 1 < W ? f[i + 1] : 0.f);
    }
}

// Segment s, (tile, item), by multiplications.
__device__ __forceinline__ tdp_seg seg_at(const tdp_geom &g, const rope_args &a, int32_t s)
{
    tdp_seg r;
    r.b = a.by_B.mod(s);
    r.t = s;
    const int32_t iW = a.by_nW.mod(s), iH = a.by_nH.mod(s), iF = s;
    const int64_t SF = g.d[0].hi[iF] - g.d[0].lo[iF];
    const int64_t SH = g.d[1].hi[iH] - g.d[1].lo[iH];
    const int64_t SW = g.d[2].hi[iW] - g.d[2].lo[iW];
    r.T = SF * SH * SW;
    r.row0 = (int64_t)g.B * tdp_tile_off(g, iF, iH, iW) + (int64_t)r.b * r.T;
    return r;
}

// HALF: element i and i + pairs are a pair, an item two vectors of W elements; otherwise elements 2 i and 2 i + 1, an item
// one vector (W even).  W is 16 bytes where rot, and half of it, allow that.  REST: a head has more than its pairs.
template <int BF16, int W, int HALF, int REST>
__global__ void __launch_bounds__(kRopeThreads)
tdp_rope_kernel(const __grid_constant__ tdp_geom g, const __grid_constant__ rope_args a)
{
    constexpr int B = W * (BF16 ? 2 : 4), U = (B + 3) / 4, P = HALF ? W : W / 2;
    tdp_pdl_trigger();
    tdp_pdl_wait();
    // segment, tile and place by multiplications: by seven divisions a thread 35840 rows of one head take 5.6 us where this takes 4.8
    int32_t seg = blockIdx.x, tr = threadIdx.x, group;
    const int32_t blk = a.by_blocks.mod(seg);
    const tdp_seg sg = seg_at(g, a, seg);
    group = a.by_team.mod(tr);
    const int64_t j = (int64_t)blk * a.rows + tr;
    if (tr >= a.rows || j >= sg.T) return;
    const int32_t item = a.by_items.mod(group);
    const int64_t row = sg.row0 + j;
    const bool turns = !REST || item < a.turned;
    // where the item's vectors lie in a head
    const int32_t o0 = turns ? item * B : (2 * a.pairs * (BF16 ? 2 : 4) + (item - a.turned) * B);
    const int32_t o1 = o0 + a.pairs * (BF16 ? 2 : 4);
    const unsigned char *x = static_cast<const unsigned char *>(a.x) + row * a.x_row + o0;
    unsigned char *out = static_cast<unsigned char *>(a.out) + row * a.out_row + o0;
    if (!turns) {
        // what lies behind the pairs is copied
        if (x == out && a.x_head == a.out_head) return;
        for (int32_t h0 = group; h0 < a.heads; h0 += 2 * kRopeAhead * a.groups) {
            uint32_t u[2 * kRopeAhead][U];
#pragma unroll
            for (int k = 0; k < 2 * kRopeAhead; ++k)
                if (h0 + k * a.groups < a.heads) load<BF16, W>(x + (h0 + k * a.groups) * a.x_head, u[k]);
#pragma unroll
            for (int k = 0; k < 2 * kRopeAhead; ++k)
                if (h0 + k * a.groups < a.heads) store<BF16, W>(out + (h0 + k * a.groups) * a.out_head, u[k]);
        }
        return;
    }
    // the first heads' loads go ahead of the sines (4096 rows of 32 heads of 128: 13.8 us for 14.8)
    uint32_t u[kRopeAhead][U], v[kRopeAhead][U];
    auto bring = [&](int32_t h0) {
#pragma unroll
        for (int k = 0; k < kRopeAhead; ++k) {
            const int32_t h = h0 + k * a.groups;
            if (h >= a.heads) break;
            load<BF16, W>(x + h * a.x_head, u[k]);
            if (HALF) load<BF16, W>(x + h * a.x_head + (o1 - o0), v[k]);
        }
    };
    bring(group);
    // cos, sin and -sin of two pairs at a time (of one where an item has one)
    constexpr int P2 = (P + 1) / 2;
    uint64_t c2[P2], s2[P2], n2[P2];
    {
        const int32_t *q = a.pos + 6 * sg.row0 + 2 * j;
        int64_t p[3];
#pragma unroll
        for (int d = 0; d < 3; ++d) {
            const int2 v = *reinterpret_cast<const int2 *>(q + 2 * d * sg.T);
            p[d] = a.middle ? (int64_t)v.x + v.y : 2 * (int64_t)v.x;
        }
        float c[2 * P2], s[2 * P2];
        c[2 * P2 - 1] = s[2 * P2 - 1] = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t f = a.table[item * P + i];
            const int32_t axis = (int32_t)f & 3;
            const uint64_t turn = (uint64_t)(f & ~3ll) * (uint64_t)(axis == 0 ? p[0] : axis == 1 ? p[1] : p[2]);
            const uint32_t t = (uint32_t)(turn >> 32);
            if (BF16) {
                const float half = (float)(int32_t)t * 0x1p-31f;        // half turns, -1 to 1
                // the fast functions, off by 2^-21 within half a turn: a thousandth of what bf16's outputs are rounded by, and a tenth of
                // the instructions (822528 rows of 8 heads of 64: 251 us for 256, 35840 rows of one head 5.2 for 5.6)
                c[i] = __cosf(half * 3.14159265f);
                s[i] = __sinf(half * 3.14159265f);
            } else {
                // the nearest quarter turn, and at most an eighth on top, which fp32 holds to 2^-28 turns; of a whole turn it holds 2^-26
                const uint32_t q = (t + 0x20000000u) >> 30;
                float p, r;
                sincospif((float)(int32_t)(t - (q << 30)) * 0x1p-31f, &r, &p);
                c[i] = q & 1 ? r : p;
                s[i] = q & 1 ? p : r;
                if ((q + 1) & 2) c[i] = -c[i];
                if (q & 2) s[i] = -s[i];
            }
            c[i] *= a.scale;
            s[i] *= a.sign * a.scale;
        }
#pragma unroll
        for (int i = 0; i < P2; ++i) {
            c2[i] = pair(c[2 * i], c[2 * i + 1]);
            s2[i] = pair(s[2 * i], s[2 * i + 1]);
            n2[i] = pair(-s[2 * i], -s[2 * i + 1]);
        }
    }
    for (int32_t h0 = group; h0 < a.heads; h0 += kRopeAhead * a.groups) {
        if (h0 > group) bring(h0);
#pragma unroll
        for (int k = 0; k < kRopeAhead; ++k) {
            const int32_t h = h0 + k * a.groups;
            if (h >= a.heads) break;
            float e[W], f[W];
            unpack<BF16, W>(u[k], e);
            if (HALF) unpack<BF16, W>(v[k], f);
#pragma unroll
            for (int i = 0; i < P2; ++i) {
                constexpr int one = P > 1;
                float none[2] = {0.f, 0.f};         // an item of one pair has no second
                float &l = HALF ? e[2 * i] : e[4 * i], &r = HALF ? f[2 * i] : e[4 * i + 1];
                float &m = one ? (HALF ? e[(2 * i + 1) * one] : e[(4 * i + 2) * one]) : none[0];
                float &q = one ? (HALF ? f[(2 * i + 1) * one] : e[(4 * i + 3) * one]) : none[1];
                const uint64_t x2 = pair(l, m), y2 = pair(r, q);
                unpair(fma2(x2, c2[i], mul2(y2, n2[i])), l, m);
                unpair(fma2(x2, s2[i], mul2(y2, c2[i])), r, q);
            }
            pack<BF16, W>(e, u[k]);
            store<BF16, W>(out + h * a.out_head, u[k]);
            if (HALF) {
                pack<BF16, W>(f, v[k]);
                store<BF16, W>(out + h * a.out_head + (o1 - o0), v[k]);
            }
        }
    }
}

tdp_status rope(tdp_plan_t plan, const tdp_rope_shape *p, const void *x, const int32_t *pos, const int64_t *table, void *out,
                float sign, tdp_stream_t stream)
{
    if (!plan || !p) return tdp_fail(TDP_ERR_INVALID_ARG, "null plan or shape");
    const tdp_geom &g = plan->g;
    if (p->heads < 1 || p->head_dim < 1 || p->rot < 2 || p->rot % 2 != 0 || p->rot > p->head_dim)
        return tdp_fail(TDP_ERR_INVALID_ARG, "need heads >= 1 and an even rot from 2 to head_dim");
    if ((p->layout != TDP_ROPE_HALF && p->layout != TDP_ROPE_INTERLEAVED) || (p->at != TDP_ROPE_START && p->at != TDP_ROPE_MIDDLE))
        return tdp_fail(TDP_ERR_INVALID_ARG, "unknown layout or place in the interval");
    if (!(p->scale - p->scale == 0.f)) return tdp_fail(TDP_ERR_INVALID_ARG, "scale must be finite");
    if (p->head_dim > TDP_MAX_ROPE_DIM || p->heads > TDP_MAX_ROPE_HEADS)
        return tdp_fail(TDP_ERR_TOO_LARGE, "head_dim above TDP_MAX_ROPE_DIM or heads above TDP_MAX_ROPE_HEADS");
    const int64_t V = 16 / g.esize, strides[4] = {p->x_row, p->x_head, p->out_row, p->out_head};
    if (p->head_dim % V != 0) return tdp_fail(TDP_ERR_MISALIGNED, "head_dim * element size must be a multiple of 16 bytes");
    for (int64_t s : strides) {
        if (s < 0) return tdp_fail(TDP_ERR_INVALID_ARG, "strides must not be negative");
        if (s % V != 0) return tdp_fail(TDP_ERR_MISALIGNED, "strides must be multiples of 16 bytes");
        if (s >= ((int64_t)1 << 38)) return tdp_fail(TDP_ERR_TOO_LARGE, "strides must be below 2^38 elements");
    }
    const int64_t R = (int64_t)g.B * g.total;
    const __int128 most = (__int128)(p->heads - 1) * std::max(p->x_head, p->out_head) + (__int128)R * std::max(p->x_row, p->out_row);
    if (most > ((__int128)1 << 56)) return tdp_fail(TDP_ERR_TOO_LARGE, "heads and rows past 2^56 elements");
    // a row's heads side by side, or a head's rows
    const __int128 D = p->head_dim, oh = p->heads > 1 ? p->out_head : D, orow = R > 1 ? p->out_row : D;
    if (!(oh >= D && (R <= 1 || orow >= (p->heads - 1) * oh + D)) && !(orow >= D && (p->heads == 1 || oh >= (R - 1) * orow + D)))
        return tdp_fail(TDP_ERR_INVALID_ARG, "out's rows and heads overlap");
    if (R == 0) return tdp_ok();
    if (!x || !pos || !table || !out) return tdp_fail(TDP_ERR_INVALID_ARG, "null x, positions, table or out");
    if (!tdp_aligned(x, 16) || !tdp_aligned(out, 16) || !tdp_aligned(pos, 8) || !tdp_aligned(table, 8))
        return tdp_fail(TDP_ERR_MISALIGNED, "heads need 16-byte, positions and table 8-byte alignment");
    if (x == out && ((p->heads > 1 && p->x_head != p->out_head) || (R > 1 && p->x_row != p->out_row)))
        return tdp_fail(TDP_ERR_INVALID_ARG, "in place with other strides");
    // the widest vector that half of rot (or rot) is a multiple of
    const int32_t half = p->layout == TDP_ROPE_HALF;
    int32_t W = (int32_t)V;
    while ((half ? p->rot / 2 : p->rot) % W != 0) W /= 2;
    rope_args a = {};
    a.x = x;
    a.pos = pos;
    a.table = table;
    a.out = out;
    a.x_row = p->x_row * g.esize;
    a.x_head = p->heads > 1 ? p->x_head * g.esize : 0;
    a.out_row = p->out_row * g.esize;
    a.out_head = p->heads > 1 ? p->out_head * g.esize : 0;
    a.heads = p->heads;
    a.pairs = p->rot / 2;
    a.turned = half ? a.pairs / W : p->rot / W;
    a.items = a.turned + (p->head_dim - p->rot) / W;
    // eight heads a thread where there are that many: its sines are made once (two heads a thread: 4096 rows of 32 heads 32 us for 15)
    a.groups = std::max(1, std::min({p->heads, kRopeThreads / a.items, (p->heads + 7) / 8}));
    a.rows = kRopeThreads / (a.items * a.groups);
    const int64_t T = tdp_max_tile_tokens(g);
    a.rows = (int32_t)std::min<int64_t>(a.rows, T);
    const int64_t blocks = (T + a.rows - 1) / a.rows;
    if (blocks * g.nt > 0x7fffffffLL / g.B) return tdp_fail(TDP_ERR_TOO_LARGE, "rotary positions: grid too large");
    a.blocks = (int32_t)blocks;
    a.middle = p->at == TDP_ROPE_MIDDLE;
    a.by_blocks = fast_div_by(a.blocks);
    a.by_team = fast_div_by(a.items * a.groups);
    a.by_items = fast_div_by(a.items);
    a.by_B = fast_div_by(g.B);
    a.by_nH = fast_div_by(g.d[1].n);
    a.by_nW = fast_div_by(g.d[2].n);
    a.sign = sign;
    a.scale = p->scale;
    const unsigned grid = (unsigned)(blocks * g.nt * g.B);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool rest = p->head_dim > p->rot;
#define TDP_ROPE(BF, W, H) \
    (rest ? tdp_launch(true, tdp_rope_kernel<BF, W, H, 1>, grid, kRopeThreads, s, g, a) : tdp_launch(true, tdp_rope_kernel<BF, W, H, 0>, grid, kRopeThreads, s, g, a))
#define TDP_ROPE2(BF, W) (half ? TDP_ROPE(BF, W, 1) : TDP_ROPE(BF, W, 0))
    cudaError_t err;
    if (g.dtype == TDP_BF16) err = W == 8 ? TDP_ROPE2(1, 8) : W == 4 ? TDP_ROPE2(1, 4) : W == 2 ? TDP_ROPE2(1, 2) : TDP_ROPE(1, 1, 1);     // odd halves alone
    else err = W == 4 ? TDP_ROPE2(0, 4) : W == 2 ? TDP_ROPE2(0, 2) : TDP_ROPE(0, 1, 1);
#undef TDP_ROPE2
#undef TDP_ROPE
    return err == cudaSuccess ? tdp_ok() : tdp_fail(TDP_ERR_CUDA, cudaGetErrorString(err));
}

}  // namespace

extern "C" tdp_status tdp_rope(tdp_plan_t plan, const tdp_rope_shape *p, const void *x, const int32_t *pos, const int64_t *table,
                               void *out, tdp_stream_t stream)
{
    return rope(plan, p, x, pos, table, out, 1.f, stream);
}

extern "C" tdp_status tdp_rope_grad(tdp_plan_t plan, const tdp_rope_shape *p, const void *dout, const int32_t *pos,
                                    const int64_t *table, void *dx, tdp_stream_t stream)
{
    return rope(plan, p, dout, pos, table, dx, -1.f, stream);
}

extern "C" tdp_status tdp_rope_table(int32_t pairs, const double *freq, const int32_t *axis, int64_t *table)
{
    if (pairs < 0 || (pairs > 0 && (!freq || !axis || !table))) return tdp_fail(TDP_ERR_INVALID_ARG, "null array or negative pairs");
    for (int32_t i = 0; i < pairs; ++i) {
        if (axis[i] < 0 || axis[i] > 2 || !(std::fabs(freq[i]) <= 0x1p20)) return tdp_fail(TDP_ERR_INVALID_ARG, "axes are 0, 1, 2 and frequencies at most 2^20");
    }
    for (int32_t i = 0; i < pairs; ++i) {
        // (start + end) / 2 is an integer times f / 4 pi turns.  The product to 106 bits, of the magnitude: the fraction of a
        // negative number would lose its last bits.
        const double f = std::fabs(freq[i]), hi = f * kInvFourPiHi, lo = std::fma(f, kInvFourPiHi, -hi) + f * kInvFourPiLo;
        const double up = std::ldexp(hi - std::floor(hi), 32), top = std::floor(up);
        const double rest = std::ldexp(up - top, 32) + std::ldexp(lo, 64);          // in 2^-64 turns
        uint64_t turns = ((uint64_t)top << 32) + (uint64_t)(int64_t)std::floor(rest + 0.5);
        turns = (freq[i] < 0 ? 0 - turns : turns) + 2;
        table[i] = (int64_t)((turns & ~3ull) | (uint64_t)axis[i]);
    }
    return tdp_ok();
}

extern "C" tdp_status tdp_rope_freqs(const int32_t *pairs, double base, int32_t scaling, double factor, double length, double *freq,
                                     int32_t *axis, float *scale)
{
    if (!pairs || !freq || !axis || !scale) return tdp_fail(TDP_ERR_INVALID_ARG, "null array");
    if (pairs[0] < 0 || pairs[1] < 0 || pairs[2] < 0) return tdp_fail(TDP_ERR_INVALID_ARG, "negative pairs");
    if ((int64_t)pairs[0] + pairs[1] + pairs[2] > TDP_MAX_ROPE_DIM / 2) return tdp_fail(TDP_ERR_TOO_LARGE, "more pairs than TDP_MAX_ROPE_DIM / 2");
    if (!(base > 0) || !std::isfinite(base) || scaling < TDP_ROPE_UNSCALED || scaling > TDP_ROPE_YARN)
        return tdp_fail(TDP_ERR_INVALID_ARG, "need a finite base > 0 and a known scaling");
    if (scaling != TDP_ROPE_UNSCALED && (!(factor >= 1) || !std::isfinite(factor))) return tdp_fail(TDP_ERR_INVALID_ARG, "need a finite factor >= 1");
    if (scaling == TDP_ROPE_YARN && (!(length > 0) || !std::isfinite(length))) return tdp_fail(TDP_ERR_INVALID_ARG, "need a finite length > 0");
    for (int32_t a = 0, at = 0; a < 3; ++a) {
        const int32_t n = pairs[a];
        const double b = scaling == TDP_ROPE_NTK && n > 1 ? base * std::pow(factor, (double)n / (n - 1)) : base;
        for (int32_t i = 0; i < n; ++i, ++at) {
            double f = std::pow(b, -(double)i / n);
            if (scaling == TDP_ROPE_LINEAR) f /= factor;
            if (scaling == TDP_ROPE_YARN) {
                const double keep = std::min(1.0, std::max(0.0, (length * f / (2 * M_PI) - 1) / (32 - 1)));
                f = f * keep + f / factor * (1 - keep);
            }
            freq[at] = f;
            axis[at] = a;
        }
    }
    *scale = scaling == TDP_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1) : 1.f;
    return tdp_ok();
}
