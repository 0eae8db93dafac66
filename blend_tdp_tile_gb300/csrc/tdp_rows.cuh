// tdp_rows.cuh -- tile-major rows as the per-tile block's operators walk them: tile t
// holds B * T_t rows (item 0's T_t tokens, then item 1's, ...) from row B*off_t on.  A
// segment is the T_t rows of one (tile, item); segment s = t * B + b.
#pragma once

#include "tdp_device.cuh"

// Division of n < 2^31 by a constant: q = n * mul >> shift, mul = ceil(2^shift / d), shift = 31 + ceil(log2 d) (T. Granlund,
// P. Montgomery, "Division by invariant integers using multiplication", PLDI 1994).  Kernels that decode a work item
// over and over use it: with n / d instead, attention of 35840 rows, 16 heads of 64, 600 of 1000 states takes 115 us for 111, of
// 168960 rows, 16 heads of 128, 512 states 544 for 533.
struct fast_div {
    uint32_t mul;
    int32_t shift, d;
    __device__ __forceinline__ int32_t div(int32_t n) const { return (int32_t)(((uint64_t)(uint32_t)n * mul) >> shift); }
    // n becomes the quotient; the remainder is returned
    __device__ __forceinline__ int32_t mod(int32_t &n) const
    {
        const int32_t q = div(n), r = n - q * d;
        n = q;
        return r;
    }
};
static inline fast_div fast_div_by(int32_t d)
{
    int32_t s = 0;
    while (((int64_t)1 << s) < d) ++s;
    fast_div f;
    f.d = d;
    f.shift = 31 + s;
    f.mul = (uint32_t)((((uint64_t)1 << f.shift) + d - 1) / d);
    return f;
}

struct tdp_seg {
    int64_t row0;      // first row
    int64_t T;         // rows
    int32_t t, b;
};

__device__ __forceinline__ tdp_seg tdp_seg_at(const tdp_geom &g, int32_t s)
{
    tdp_seg r;
    r.t = s / g.B;
    r.b = s - r.t * g.B;
    const int32_t nW = g.d[2].n, nH = g.d[1].n;
    const int32_t iW = r.t % nW, iH = (r.t / nW) % nH, iF = r.t / (nW * nH);
    const int64_t SF = g.d[0].hi[iF] - g.d[0].lo[iF];
    const int64_t SH = g.d[1].hi[iH] - g.d[1].lo[iH];
    const int64_t SW = g.d[2].hi[iW] - g.d[2].lo[iW];
    r.T = SF * SH * SW;
    r.row0 = (int64_t)g.B * tdp_tile_off(g, iF, iH, iW) + (int64_t)r.b * r.T;
    return r;
}

// Rows of the largest segment (host).
static inline int64_t tdp_max_tile_tokens(const tdp_geom &g)
{
    int64_t m = 1;
    for (int d = 0; d < 3; ++d) {
        int32_t s = 0;
        for (int32_t i = 0; i < g.d[d].n; ++i)
            if (g.d[d].hi[i] - g.d[d].lo[i] > s) s = g.d[d].hi[i] - g.d[d].lo[i];
        m *= s;
    }
    return m;
}

// Element type of a plan's dtype and its 16-byte vectors as fp32.
template <int BF16>
struct tdp_elem {
    using type = float;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *f)
    {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

template <>
struct tdp_elem<1> {
    using type = __nv_bfloat16;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *f)
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = tdp_bf16_lo(w[i]);
            f[2 * i + 1] = tdp_bf16_hi(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        return make_uint4(tdp_pack_bf16x2(f[0], f[1]), tdp_pack_bf16x2(f[2], f[3]), tdp_pack_bf16x2(f[4], f[5]),
                          tdp_pack_bf16x2(f[6], f[7]));
    }
};
