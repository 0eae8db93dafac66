"""Plain 64-bit forms of the per-tile block's operators, for the tests: numpy loops over (tile, item)
segments, sharing no code with the library.  Each returns the values and, for every value, the sum
of the magnitudes of the terms it is made of: a rounding of relative size u anywhere in the computation moves a value by
at most a few u times that sum, so tolerances are multiples of it and not of the value."""
import math

import numpy as np


def boxes(L, n, o):
    o = o if n > 1 else 0
    c = [i * L // n for i in range(n + 1)]
    return [(c[i] - (o // 2 if i else 0), c[i + 1] + (o - o // 2 if i < n - 1 else 0)) for i in range(n)]


def segments(B, dims, tiles, overlap):
    """[(tile, item, first row, rows)] of the tile-major rows."""
    out, row, t = [], 0, 0
    b = [boxes(*a) for a in zip(dims, tiles, overlap)]
    for f in b[0]:
        for h in b[1]:
            for w in b[2]:
                T = (f[1] - f[0]) * (h[1] - h[0]) * (w[1] - w[0])
                for i in range(B):
                    out.append((t, i, row, T))
                    row += T
                t += 1
    return out, row


def xattn(segs, q, k, v, mask, scale, dout=None):
    """out, lse (and dq, dk, dv) as {name: (value, magnitude)}; mask None, [B,S] or [nt,B,S]."""
    R, H, D = q.shape
    B, S, K, _ = k.shape
    G = H // K
    z = lambda *s: np.zeros(s)  # noqa: E731
    r = {"out": (z(R, H, D), z(R, H, D)), "lse": (np.full((R, H), -math.inf), z(R, H))}
    if dout is not None:
        r |= {"dq": (z(R, H, D), z(R, H, D)), "dk": (z(B, S, K, D), z(B, S, K, D)), "dv": (z(B, S, K, D), z(B, S, K, D))}
    smax = 0.0
    for t, b, r0, T in segs:
        on = np.arange(S) if mask is None else np.flatnonzero(mask[t, b] if mask.ndim == 3 else mask[b])
        if not len(on):
            continue
        rows = slice(r0, r0 + T)
        for h in range(H):
            x, kk, vv = q[rows, h], k[b, on, h // G], v[b, on, h // G]
            s = scale * x @ kk.T
            sa = abs(scale) * np.abs(x) @ np.abs(kk).T
            smax = max(smax, float(sa.max()))
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            l = e.sum(1, keepdims=True)
            p = e / l
            r["lse"][0][rows, h] = (top + np.log(l))[:, 0]
            r["lse"][1][rows, h] = sa.max(1) + np.abs(top[:, 0]) + 1
            o = p @ vv
            r["out"][0][rows, h], r["out"][1][rows, h] = o, p @ np.abs(vv)
            if dout is None:
                continue
            g = dout[rows, h]
            ds = p * (g @ vv.T - (g * o).sum(1, keepdims=True)) * scale
            dsa = p * (np.abs(g) @ np.abs(vv).T + (np.abs(g) * (p @ np.abs(vv))).sum(1, keepdims=True)) * abs(scale)
            r["dq"][0][rows, h], r["dq"][1][rows, h] = ds @ kk, dsa @ np.abs(kk)
            for name, a, aa in (("dk", ds.T @ x, dsa.T @ np.abs(x)), ("dv", p.T @ g, p.T @ np.abs(g))):
                r[name][0][b, on, h // G] += a
                r[name][1][b, on, h // G] += aa
    return r, smax


def xattn_unit(dtype, D, smax):
    """Relative size of the roundings in cross attention, against the magnitudes of xattn().

    fp32: a score is off by up to D * 2^-24 of its magnitude sum (smax at most), its exponential by that
    and a few 2^-24 more, and so is every sum of products.  bf16 (8 significant bits: 2^-8) besides rounds each
    probability or gradient of a score once, out once where delta reads it, and the result: 3 * 2^-8 in all."""
    u = 2.0 ** -24 * (4 * D * smax + 2 * D + 64)
    return u + (3 * 2.0 ** -8 if dtype == "bf16" else 0.0)


def gnorm(segs, nt, B, x, G, gamma, beta, eps, silu, dy=None):
    R, C = x.shape
    cg = C // G
    z = lambda *s: np.zeros(s)  # noqa: E731
    r = {"y": (z(R, C), z(R, C)), "mean": (z(nt, B, G), z(nt, B, G)), "rstd": (z(nt, B, G), z(nt, B, G))}
    if dy is not None:
        r |= {"dx": (z(R, C), z(R, C)), "dgamma": (z(C), z(C)), "dbeta": (z(C), z(C))}
    for t, b, r0, T in segs:
        rows = slice(r0, r0 + T)
        xs = x[rows].reshape(T, G, cg)
        mu = xs.mean((0, 2))
        dev = xs - mu[:, None]
        var = (dev ** 2).mean((0, 2))
        rs = 1 / np.sqrt(var + eps)
        big = np.abs(xs).max((0, 2))
        r["mean"][0][t, b], r["mean"][1][t, b] = mu, big
        # a mean off by u * big moves the variance by u * big * std, and rstd by half that over the variance
        r["rstd"][0][t, b], r["rstd"][1][t, b] = rs, rs * (1 + big * rs)
        h = (dev * rs[:, None]).reshape(T, C)
        # the mean is off by u * big wherever x is, near the mean too
        ha = ((np.abs(xs) + big[:, None]) * rs[:, None] + np.abs(h.reshape(T, G, cg)) * (big * rs)[:, None]).reshape(T, C)
        zz = h * gamma + beta
        za = ha * np.abs(gamma) + np.abs(beta)
        s = 1 / (1 + np.exp(-zz)) if silu else 1.0
        r["y"][0][rows], r["y"][1][rows] = zz * s, za * 1.2          # |silu'| <= 1.1
        if dy is None:
            continue
        slope = s * (1 + zz * (1 - s)) if silu else 1.0
        d = dy[rows] * slope
        da = np.abs(dy[rows]) * (1.2 + (za if silu else 0))            # |silu''| <= 0.5
        r["dgamma"][0][:] += (d * h).sum(0)
        r["dgamma"][1][:] += (da * ha).sum(0)
        r["dbeta"][0][:] += d.sum(0)
        r["dbeta"][1][:] += da.sum(0)
        e, ea = (d * gamma).reshape(T, G, cg), (da * np.abs(gamma)).reshape(T, G, cg)
        hg, hag = h.reshape(T, G, cg), ha.reshape(T, G, cg)
        m1, m2 = e.mean((0, 2)), (e * hg).mean((0, 2))
        m1a, m2a = ea.mean((0, 2)), (ea * hag).mean((0, 2))
        k = rs[:, None]
        r["dx"][0][rows] = (k * (e - m1[:, None] - hg * m2[:, None])).reshape(T, C)
        r["dx"][1][rows] = (k * (1 + (big * rs)[:, None]) * (ea + m1a[:, None] + hag * m2a[:, None])).reshape(T, C)
    return r


def philox(n, seed, offset):
    """Word i of the dropout generator for i < n: word i % 4 of Philox4x32-10, counter {i / 4, offset}."""
    i = np.arange((n + 3) // 4, dtype=np.uint64)
    return philox_at(i, seed, offset).reshape(-1)[:n]


def philox_at(i, seed, offset):
    m32 = np.uint64(0xFFFFFFFF)
    i = np.asarray(i, np.uint64)
    c = [i & m32, i >> np.uint64(32), np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & m32, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & m32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1)
