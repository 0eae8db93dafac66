"""Plain 64-bit forms of the norm, the 8-bit products and the rotary positions, for the tests: numpy, sharing no code with the
library."""
import math

import numpy as np

LEAST = 2.0 ** -100
U32 = 2.0 ** -24            # half a step of fp32, relative


def e4m3(v):
    """The nearest of e4m3's values, the even one of two: steps of 2^(e-3) from 2^e on, of 2^-9 below 2^-6; 448 at most."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 448.0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.rint(a / step) * step, v)


def half_step8(v):
    """Half a step of e4m3 at |v|: 2^-4 of it, or 2^-10."""
    return np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10)


def rows8(x):
    """Values before their rounding to e4m3, and the scales."""
    top = np.maximum(np.abs(x).max(-1), LEAST)
    return x * 448 / top[..., None], top / 448


def rms_norm(h, w, eps):
    rstd = (np.mean(h * h, -1) + eps) ** -0.5
    u = h * rstd[:, None]
    return rstd, u, u * w


def rms_norm_grad(u, rstd, w, dy, dh):
    g = dy * w
    dx = rstd[:, None] * (g - u * (g * u).mean(-1, keepdims=True)) + dh
    size = rstd[:, None] * (np.abs(g) + np.abs(u) * np.abs(g * u).mean(-1, keepdims=True)) + np.abs(dh)
    return dx, size, (dy * u).sum(0), np.abs(dy * u).sum(0)


def angles(segs, Q, freq, axis, middle):
    """[R, pairs] radians; Q tile-major int32."""
    rows = sum(T for *_, T in segs)
    pos = np.zeros((rows, 3))
    for _, _, r0, T in segs:
        p = Q[6 * r0:6 * (r0 + T)].reshape(3, T, 2).astype(np.float64)
        pos[r0:r0 + T] = (p.mean(-1) if middle else p[..., 0]).T
    return pos, pos[:, axis] * freq


def turn(x, angle, scale, interleaved, back=False):
    """[R, H, D] turned, and the magnitudes of what was added."""
    n = angle.shape[1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    c, s = scale * np.cos(angle)[:, None], scale * np.sin(-angle if back else angle)[:, None]
    y, size = x.copy(), np.abs(x)
    for to, v, m in ((0, a * c - b * s, np.abs(a) + np.abs(b)), (1, a * s + b * c, np.abs(a) + np.abs(b))):
        at = slice(to, 2 * n, 2) if interleaved else slice(to * n, to * n + n)
        y[..., at], size[..., at] = v, m * abs(scale)
    return y, size


def yarn(n, base, factor, length):
    f = [base ** (-i / n) for i in range(n)]
    keep = [min(1, max(0, (length * v / (2 * math.pi) - 1) / 31)) for v in f]
    return [v * k + v / factor * (1 - k) for v, k in zip(f, keep)]
