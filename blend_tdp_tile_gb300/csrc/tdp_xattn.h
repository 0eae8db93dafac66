// tdp_xattn.h -- what the cross-attention kernels and their entry points share.
//
// The rows a kernel works on are "packed": within a segment and a key head, packed row
// r = token * G + j is query head kvh * G + j of that token (G query heads share a key head),
// so that all rows of a block read the same keys.  With one batch item and a mask that is the same for
// every tile, all tiles are one segment.
#pragma once

#include "tdp_internal.h"
#include "tdp_rows.cuh"

struct xattn_args {
    const void *q, *k, *v;
    const uint8_t *mask;
    const void *o;              // gradient: the forward's out
    const void *dout;
    void *out, *dq, *dk, *dv;
    float *lse;                 // written by the forward (may be NULL), read by the gradient
    float *delta;               // [R, Hq] gradient: dout . out
    int32_t *kept_n;            // bf16: [mask rows] kept 128-state tiles, their indexes and the masks of their states
    int32_t *kept_states;       //       [mask rows] states in them
    int32_t *kept_tile;         //       [mask rows, tiles]
    uint4 *kept_words;          //       [mask rows, tiles]
    uint4 *state_words;         //       masks of every tile's states [mask rows, tiles] (gradient)
    float *po, *pl;             // forward split over states: partial out [split][R, Hq, D] and lse [split][R, Hq]
    float *pk, *pv;             // gradient split over rows: partial dk, dv [split][B, S, Hkv, D]
    float *pq;                  // fp32 gradient split over states: partial dq [qsplit][R, Hq, D]
    int64_t q_row, q_head, k_item, k_state, k_head, v_item, v_state, v_head;
    int64_t rows;               // R
    int32_t Hq, Hkv, G, D, S;
    // bf16: rows of a 128-row tile are Gp query heads of TT = 128 / Gp tokens, Gp the largest divisor of G up to 128
    int32_t Gp, TT;
    fast_div by_blocks, by_heads, by_split, by_B, by_nH, by_nW, by_group;      // head blocks: Hq / Gp; by_group: G
    int32_t flat;               // all tiles are one segment
    int32_t per_tile;           // mask row per segment, else per item
    int32_t segs;               // segments
    int32_t blocks;             // row blocks of the largest segment
    int32_t split;              // parts the states (forward) or the row blocks (dk, dv) are split into
    int32_t part;               // fp32: 64-state tiles (forward) or row blocks (dk, dv) of a part
    int32_t qsplit, qpart;      // fp32: parts the states are split into for dq, 64-state tiles of a part
    float scale;
};

// Segment s of the walk: a (tile, item), or everything.
__device__ __forceinline__ tdp_seg xattn_seg(const tdp_geom &g, const xattn_args &a, int32_t s)
{
    if (a.flat) {
        tdp_seg r;
        r.row0 = 0;
        r.T = a.rows;
        r.t = r.b = 0;
        return r;
    }
    return tdp_seg_at(g, s);
}

// The same by multiplications (bf16 kernels).
__device__ __forceinline__ tdp_seg xattn_seg_fast(const tdp_geom &g, const xattn_args &a, int32_t s)
{
    tdp_seg r;
    if (a.flat) {
        r.row0 = 0;
        r.T = a.rows;
        r.t = r.b = 0;
        return r;
    }
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

__device__ __forceinline__ const uint8_t *xattn_mask(const xattn_args &a, const tdp_geom &g, const tdp_seg &seg)
{
    return a.mask ? a.mask + (a.per_tile ? (int64_t)seg.t * g.B + seg.b : seg.b) * (int64_t)a.S : nullptr;
}
