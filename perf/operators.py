"""Cases for the operators a per-tile transformer block runs between the tile split and the blend.

Three operators, each over the plan's tile-major rows (tile t holds B * T_t rows, item after item):

  xattn    cross attention of the tiles' tokens to an encoder's states (forward; forward and gradients)
  gn       group normalisation of every (tile, item), channels last, with SiLU (forward; forward and gradients)
  dropout  residual + dropout from a counter-based generator, its mask never stored (forward and gradient)

`run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once at the end),
or, where `own` is true, through the package's entry points.  `exact` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------- cases
def _plan(B, F, H, W, nf=1, nh=1, nw=1, of=0, oh=0, ow=0):
    return dict(B=B, F=F, H=H, W=W, nf=nf, nh=nh, nw=nw, of=of, oh=oh, ow=ow)


TINY = _plan(1, 3, 8, 12, 1, 2, 2, 0, 2, 2)            # the repository's workloads
SMALL = _plan(1, 16, 32, 48, 1, 2, 2, 0, 8, 8)
MEDIUM = _plan(1, 16, 64, 96, 1, 4, 4, 0, 8, 8)
TEMPORAL = _plan(2, 32, 68, 120, 2, 3, 3, 4, 8, 8)
LARGE = _plan(1, 64, 128, 192, 2, 8, 8, 4, 16, 16)
RAGGED = _plan(2, 9, 17, 30, 2, 2, 2, 2, 4, 4)         # odd extents: tiles of many sizes
TOKEN = _plan(8, 1, 1, 1)                              # one token per item


def _xattn(name, plan, dtype, heads, kv_heads, dim, keys, mask, kept, train, fused):
    return dict(name=name, op="xattn", dtype=dtype, heads=heads, kv_heads=kv_heads, dim=dim, keys=keys,
                mask=mask, kept=kept, train=train, fused=fused, **plan)


def _gn(name, plan, dtype, channels, groups, train):
    return dict(name=name, op="gn", dtype=dtype, channels=channels, groups=groups, train=train, **plan)


def _dropout(name, dtype, n, p):
    return dict(name=name, op="dropout", dtype=dtype, n=n, p=p)


def listed():
    return [
        # one query token per item against long, padded encoder states: the serving step of an untiled stream
        _xattn("xattn token bf16", TOKEN, "bf16", 32, 8, 128, 8192, "length", 0.9, False, True),
        # the smallest problem the repository has, a short prompt: latency counts
        _xattn("xattn tiny f32", TINY, "f32", 4, 4, 32, 77, "none", 1.0, False, False),
        # a padded prompt (states on the right) at the small latent
        _xattn("xattn small bf16", SMALL, "bf16", 16, 16, 64, 1000, "left", 0.6, False, True),
        # the whole tile set of the medium latent against a full prompt: the largest forward
        _xattn("xattn medium bf16", MEDIUM, "bf16", 16, 16, 128, 512, "none", 1.0, False, False),
        # training with heads shared in groups of four
        _xattn("xattn train shared bf16", SMALL, "bf16", 16, 4, 128, 640, "length", 1.0, True, False),
        # training on tiles of many sizes, each tile seeing the conditioning tokens that it keeps
        _xattn("xattn train ragged bf16", RAGGED, "bf16", 6, 6, 80, 1024, "keep", 0.5, True, False),
        # the smallest latent: latency counts
        _gn("gn tiny f32", TINY, "f32", 16, 4, False),
        # the largest tile set, forward
        _gn("gn large bf16", LARGE, "bf16", 128, 32, False),
        # training at two items and eighteen tiles
        _gn("gn train temporal bf16", TEMPORAL, "bf16", 128, 32, True),
        # training with groups that end inside a 16-byte vector, tiles of many sizes
        _gn("gn train ragged f32", RAGGED, "f32", 120, 20, True),
        # a block's residual at the temporal tile set
        _dropout("dropout temporal bf16", "bf16", 2 * 36 * 84 * 136 * 128, 0.1),
        # an odd number of elements
        _dropout("dropout odd f32", "f32", 420 * 129 + 1, 0.25),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_dim(rng, most):
    L = _loguniform(rng, 1, most)
    n = rng.randint(1, min(L, 4))
    return L, n, rng.randint(0, L // n) if n > 1 else 0


def _draw_plan(rng, cells):
    f, h, w = _draw_dim(rng, 24), _draw_dim(rng, 72), _draw_dim(rng, 96)
    if rng.random() < 0.1:
        f = h = w = (1, 1, 0)
    B = rng.choice([1, 1, 2, 3])
    p = _plan(B, f[0], h[0], w[0], f[1], h[1], w[1], f[2], h[2], w[2])
    return p if _geometry(p)[3] * B <= cells else _draw_plan(rng, cells)


def draw(rng):
    op = rng.choice(["xattn", "xattn", "gn", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "dropout":
        return dict(op=op, dtype=dtype, n=_loguniform(rng, 1000, 100_000_000), p=round(rng.uniform(0.0, 0.6), 3))
    if op == "gn":
        unit = 16 // ESIZE[dtype]
        C = unit * _loguniform(rng, 2, 64)
        p = _draw_plan(rng, 60_000_000 // C)
        # of fewer than 32 values normalised together a gradient is little more than rounding
        train = rng.random() < 0.5
        groups = [g for g in (1, 2, 4, 8, 16, 20, 32) if C % g == 0 and (not train or _geometry(p)[0].min() * (C // g) >= 32)]
        return dict(op=op, dtype=dtype, channels=C, groups=rng.choice(groups or [1]), train=train and bool(groups), **p)
    train = rng.random() < 0.5
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 1, 2, 4])
    dim = rng.choice([32, 40, 64, 64, 80, 112, 128, 128])
    keys = _loguniform(rng, 4 if train else 1, 3000)
    most = (7e11 if dtype == "bf16" else 5e10) / (14 if train else 4)
    p = _draw_plan(rng, min(most / (heads * dim * keys), 2e9 / (heads * keys), 1e8 / (heads * dim)))
    mask = rng.choice(["none", "length", "left", "keep"])
    return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv, dim=dim, keys=keys, mask=mask,
                kept=1.0 if mask == "none" else round(rng.uniform(0.05, 1.0), 3), train=train, fused=rng.random() < 0.5, **p)


# ---------------------------------------------------------------- geometry
def _boxes(L, n, o):
    i = np.arange(n)
    o = o if n > 1 else 0
    lo = np.where(i > 0, i * L // n - o // 2, 0)
    hi = np.where(i < n - 1, (i + 1) * L // n + o - o // 2, L)
    return hi - lo


def _geometry(c):
    """Tokens per tile [nt], token offset per tile [nt], tile of each token [tot], tokens in all."""
    s = [_boxes(c["F"], c["nf"], c["of"]), _boxes(c["H"], c["nh"], c["oh"]), _boxes(c["W"], c["nw"], c["ow"])]
    T = (s[0][:, None, None] * s[1][None, :, None] * s[2][None, None, :]).reshape(-1).astype(np.int64)
    off = np.cumsum(T) - T
    return T, off, np.repeat(np.arange(len(T)), T), int(T.sum())


def _rows(c):
    """Row of token u (of all tiles) of item b in the tile-major buffers: [B, tot]."""
    T, off, tile, tot = _geometry(c)
    u = np.arange(tot)
    b = np.arange(c["B"])[:, None]
    return c["B"] * off[tile] + b * T[tile] + (u - off[tile])


def _kept(c):
    """Keys that item b keeps: two at least, so that a gradient is more than rounding; the last of several items of a
    masked case keeps none where it is trained."""
    k = np.maximum(2, np.round(c["keys"] * c["kept"] * (1 - 0.5 * np.arange(c["B"]) / c["B"])).astype(np.int64))
    if c["train"] and c["B"] > 1 and c["mask"] != "none":
        k[-1] = 0
    return np.minimum(k, c["keys"]) if c["mask"] != "none" else np.full(c["B"], c["keys"])


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)

    s = {"case": case}
    if case["op"] == "dropout":
        n = case["n"]
        s |= {"x": normal(n), "res": normal(n, std=3.0), "dout": normal(n, std=0.01),
              "rng": torch.randint(0, 1 << 62, (2,), generator=g, device="cuda", dtype=torch.int64)}
        if own:
            s |= {"plan": _own_plan(dict(TINY, dtype=case["dtype"])), "out": torch.empty_like(s["x"]), "dx": torch.empty_like(s["x"])}
        return s
    T, off, tile, tot = _geometry(case)
    R, B = case["B"] * tot, case["B"]
    s |= {"rows": torch.from_numpy(_rows(case)).cuda(), "tile": torch.from_numpy(tile).cuda()}
    if case["op"] == "gn":
        C, G, nt = case["channels"], case["groups"], len(T)
        # activations of a convolution: channels with means and scales of their own
        level = torch.randn((C,), generator=g, device="cuda") * 0.5
        size = torch.rand((C,), generator=g, device="cuda") * 1.5 + 0.25
        s |= {"x": (torch.randn((R, C), generator=g, device="cuda") * size + level).to(dt),
              "gamma": normal(C, std=0.2, mean=1.0), "beta": normal(C, std=0.2)}
        j = np.arange(T.max())
        start = (B * off[:, None] + np.arange(B) * T[:, None]).reshape(-1)
        size = np.repeat(T, B)
        s |= {"pad": torch.from_numpy(start[:, None] + np.minimum(j, size[:, None] - 1)).cuda(),
              "in": torch.from_numpy(j < size[:, None]).cuda(), "size": torch.from_numpy(size).cuda()}
        if case["train"]:
            s["dy"] = normal(R, C, std=0.01)
        if own:
            f32 = dict(dtype=torch.float32, device="cuda")
            s |= {"plan": _own_plan(case), "y": torch.empty_like(s["x"]),
                  "mean": torch.empty((nt, B, G), **f32), "rstd": torch.empty((nt, B, G), **f32),
                  "dx": torch.empty_like(s["x"]), "dgamma": torch.empty(C, **f32), "dbeta": torch.empty(C, **f32)}
        return s
    S, H, K, D = case["keys"], case["heads"], case["kv_heads"], case["dim"]
    s["q"] = normal(R, H, D)
    if case["fused"]:  # keys and values side by side, as one projection writes them
        kv = normal(B, S, 2, K, D)
        s |= {"k": kv[:, :, 0], "v": kv[:, :, 1]}
    else:
        s |= {"k": normal(B, S, K, D), "v": normal(B, S, K, D)}
    s["mask"] = None
    kept = torch.from_numpy(_kept(case)).cuda()
    at = torch.arange(S, device="cuda")
    if case["mask"] == "length":
        s["mask"] = at < kept[:, None]
    elif case["mask"] == "left":
        s["mask"] = at >= S - kept[:, None]
    elif case["mask"] == "keep":  # a run of tokens from a place of each tile's own
        first = torch.randint(0, S, (len(T), B, 1), generator=g, device="cuda")
        s["mask"] = (at - first) % S < kept[:, None]
    if s["mask"] is not None:  # what lies in the padding is not defined
        gone = ~s["mask"].reshape(-1, B, S).any(0)
        s["k"].masked_fill_(gone[:, :, None, None], float("nan"))
        s["v"].masked_fill_(gone[:, :, None, None], float("inf"))
    if case["train"]:
        s["dout"] = normal(R, H, D, std=0.01)
    if own:
        s |= {"plan": _own_plan(case), "out": torch.empty_like(s["q"]),
              "lse": torch.empty((R, H), dtype=torch.float32, device="cuda") if case["train"] else None}
        if case["train"]:
            s |= {"dq": torch.empty_like(s["q"]), "dk": torch.empty((B, S, K, D), dtype=dt, device="cuda"),
                  "dv": torch.empty((B, S, K, D), dtype=dt, device="cuda")}
    return s


def _own_plan(c):
    import blend_tdp_tile_gb300 as tdp
    return tdp.tdp_plan_create(c["B"], c["F"], c["H"], c["W"], 8, c["dtype"],
                               (c["nf"], c["nh"], c["nw"]), (c["of"], c["oh"], c["ow"]))


# ---------------------------------------------------------------- one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_xattn(s):
    import blend_tdp_tile_gb300 as tdp
    tdp.tdp_cross_attn(s["plan"], s["q"], s["k"], s["v"], s["mask"], s["out"], s["lse"])
    if not s["case"]["train"]:
        return s["out"]
    tdp.tdp_cross_attn_grad(s["plan"], s["q"], s["k"], s["v"], s["mask"], s["out"], s["lse"], s["dout"],
                            s["dq"], s["dk"], s["dv"])
    return {"out": s["out"], "lse": s["lse"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _own_gn(s):
    import blend_tdp_tile_gb300 as tdp
    G = s["case"]["groups"]
    tdp.tdp_group_norm(s["plan"], s["x"], G, s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], act="silu")
    r = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if s["case"]["train"]:
        tdp.tdp_group_norm_grad(s["plan"], s["x"], G, s["gamma"], s["beta"], s["mean"], s["rstd"], s["dy"],
                                s["dx"], s["dgamma"], s["dbeta"], act="silu")
        r |= {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    return r


def _own_dropout(s):
    import blend_tdp_tile_gb300 as tdp
    p = s["case"]["p"]
    tdp.tdp_dropout_add(s["plan"], s["x"], s["res"], p, s["rng"], s["out"])
    tdp.tdp_dropout_grad(s["plan"], s["dout"], p, s["rng"], s["dx"])
    return {"out": s["out"], "dx": s["dx"]}


def _plain_xattn(s):
    c = s["case"]
    B, S, H, K, D, dt = c["B"], c["keys"], c["heads"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]]
    rows, N, G = s["rows"], s["rows"].shape[1], H // K
    scale = 1 / math.sqrt(D)

    def by_item(x):  # [R, H, D] -> [B, K, N * G, D]
        return x[rows].float().reshape(B, N, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, N * G, D)

    def to_rows(x):  # back, rounded
        y = torch.empty_like(s["q"])
        y[rows] = x.reshape(B, K, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H, D).to(dt)
        return y

    q, k, v = by_item(s["q"]), s["k"].float().permute(0, 2, 1, 3), s["v"].float().permute(0, 2, 1, 3)
    if s["mask"] is not None:
        seen = s["mask"].reshape(-1, B, S).any(0)[:, None, :, None]
        k, v = torch.where(seen, k, 0), torch.where(seen, v, 0)
    p = q @ k.transpose(-1, -2) * scale
    if s["mask"] is not None:
        m = s["mask"].expand(c["nf"] * c["nh"] * c["nw"], B, S)[s["tile"]].transpose(0, 1)
        p = p.reshape(B, K, N, G, S).masked_fill_(~m[:, None, :, None, :], -math.inf).reshape(B, K, N * G, S)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    p = (p - top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, 1, total)
    out = p @ v
    if not c["train"]:
        return to_rows(out)
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    lse[rows] = (top + total.log()).reshape(B, K, N, G).transpose(1, 2).reshape(B, N, H)
    dout = by_item(s["dout"])
    dv = p.transpose(-1, -2) @ dout
    ds = p * (dout @ v.transpose(-1, -2) - (dout * out).sum(-1, keepdim=True)) * scale
    return {"out": to_rows(out), "lse": lse, "dq": to_rows(ds @ k),
            "dk": (ds.transpose(-1, -2) @ q).transpose(1, 2).to(dt), "dv": dv.transpose(1, 2).to(dt)}


def _plain_gn(s):
    c = s["case"]
    C, G, dt = c["channels"], c["groups"], DTYPES[c["dtype"]]
    here, pad, eps = s["in"][:, :, None, None], s["pad"], 1e-5
    n = (s["size"] * (C // G)).float()[:, None]

    def segments(x):  # [R, C] -> [nt * B, Tmax, G, C / G], zero where a tile has ended
        return torch.where(here, x[pad].float().reshape(*pad.shape, G, C // G), 0)

    def to_rows(x):
        y = torch.empty_like(s["x"])
        y[pad[s["in"]]] = x.reshape(*pad.shape, C)[s["in"]].to(dt)
        return y

    x = segments(s["x"])
    mean = x.sum((1, 3)) / n
    x = torch.where(here, x - mean[:, None, :, None], 0)
    rstd = 1 / torch.sqrt(x.square().sum((1, 3)) / n + eps)
    xhat = x.mul_(rstd[:, None, :, None])
    gamma, beta = s["gamma"].float().reshape(G, C // G), s["beta"].float().reshape(G, C // G)
    z = xhat * gamma + beta
    sig = 1 / (1 + torch.exp(-z))
    shape = (c["nf"] * c["nh"] * c["nw"], c["B"], G)
    r = {"y": to_rows(z * sig), "mean": mean.reshape(shape), "rstd": rstd.reshape(shape)}
    if c["train"]:
        dz = segments(s["dy"]) * sig * (1 + z * (1 - sig))
        r |= {"dgamma": (dz * xhat).sum((0, 1)).reshape(C), "dbeta": dz.sum((0, 1)).reshape(C)}
        dz = dz * gamma
        a, b = dz.sum((1, 3)) / n, (dz * xhat).sum((1, 3)) / n
        r["dx"] = to_rows((dz - a[:, None, :, None] - xhat * b[:, None, :, None]) * rstd[:, None, :, None])
    return r


def _mulhilo(a, m):
    """High and low 32 bits of a * m; a holds 32-bit values in 64 bits."""
    p = a * m  # wraps past 2^63: the low 64 bits are right
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _philox_round(state, r, k0, k1):
    """One round of Philox4x32 (Salmon, Moraes, Dror, Shaw, 2011), its key bumped r times."""
    h0, l0 = _mulhilo(state[0], 0xD2511F53)
    h1, l1 = _mulhilo(state[2], 0xCD9E8D57)
    return h1 ^ state[1] ^ ((k0 + r * 0x9E3779B9) & 0xFFFFFFFF), l1, h0 ^ state[3] ^ ((k1 + r * 0xBB67AE85) & 0xFFFFFFFF), l0


def _plain_words(n, rng):
    """Word i of the generator for each element i < n: word i % 4 of Philox4x32-10 of counter (i / 4, rng[1]) and key rng[0]."""
    at = torch.arange((n + 3) // 4, device=rng.device)
    k0, k1 = rng[0] & 0xFFFFFFFF, (rng[0] >> 32) & 0xFFFFFFFF
    x = (at & 0xFFFFFFFF, at >> 32, (rng[1] & 0xFFFFFFFF).expand_as(at), ((rng[1] >> 32) & 0xFFFFFFFF).expand_as(at))
    for r in range(10):
        x = _philox_round(x, r, k0, k1)
    return torch.stack(x, 1).reshape(-1)[:n]


def _plain_dropout(s):
    c = s["case"]
    dt, keep = DTYPES[c["dtype"]], _plain_words(c["n"], s["rng"]) >= round(c["p"] * 2**32)
    scale = 1 / (1 - c["p"])
    return {"out": (s["res"].float() + torch.where(keep, s["x"].float() * scale, 0)).to(dt),
            "dx": torch.where(keep, s["dout"].float() * scale, 0).to(dt)}


_plain = {"xattn": _plain_xattn, "gn": _plain_gn, "dropout": _plain_dropout}
_own = {"xattn": _own_xattn, "gn": _own_gn, "dropout": _own_dropout}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = ESIZE[case["dtype"]]
    if case["op"] == "dropout":  # x, res -> out; dout -> dx
        return {"bytes": 5 * e * case["n"], "flops": 3 * case["n"]}
    T, _, _, tot = _geometry(case)
    R = case["B"] * tot
    if case["op"] == "gn":  # x -> y; with the gradients x, dy -> dx
        n = R * case["channels"]
        stats = 8 * len(T) * case["B"] * case["groups"]
        return {"bytes": e * n * (4 if case["train"] else 2) + stats, "flops": n * (40 if case["train"] else 12)}
    D, H, K = case["dim"], case["heads"], case["kv_heads"]
    kept = _kept(case)
    pairs = tot * int(kept.sum())
    seen = case["B"] * case["keys"] if case["mask"] == "keep" else int(kept.sum())
    q, kv = R * H * D * e, seen * K * D * e
    mask = 0 if case["mask"] == "none" else case["keys"] * case["B"] * (len(T) if case["mask"] == "keep" else 1)
    if not case["train"]:  # q, k, v -> out: two products
        return {"bytes": 2 * q + 2 * kv + mask, "flops": 4 * D * H * pairs}
    # q, k, v, dout -> out, lse, dq, dk, dv: seven products
    return {"bytes": 4 * q + 2 * kv + 2 * case["B"] * case["keys"] * K * D * e + 4 * R * H + mask, "flops": 14 * D * H * pairs}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        return _exact_dropout(case, s)
    T, off, _, _ = _geometry(case)
    B = case["B"]
    segs = [(t, b, slice(B * int(off[t]) + b * int(T[t]), B * int(off[t]) + (b + 1) * int(T[t]))) for t in range(len(T)) for b in range(B)]
    return _exact_gn(case, s, segs) if case["op"] == "gn" else _exact_xattn(case, s, segs)


def _exact_dropout(c, s):
    """The generator in halves of 16 bits, so that no product wraps."""
    n, (seed, offset) = c["n"], [int(v) for v in s["rng"].cpu()]
    low = 0xFFFF

    def product(a, m):
        a0, a1, m0, m1 = a & low, a >> 16, m & low, m >> 16
        mid = a1 * m0 + (a0 * m0 >> 16)
        mid2 = a0 * m1 + (mid & low)
        return a1 * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 & low) << 16) | (a0 * m0 & low)

    out, dx = torch.empty(n, dtype=torch.float64, device="cuda"), torch.empty(n, dtype=torch.float64, device="cuda")
    step = 1 << 24
    for a in range(0, n, 4 * step):
        count = min(step, (n - a + 3) // 4)
        i = torch.arange(a // 4, a // 4 + count, device="cuda")
        w = [i % 2**32, i // 2**32, torch.full_like(i, offset % 2**32), torch.full_like(i, offset // 2**32 % 2**32)]
        key = [seed % 2**32, seed // 2**32 % 2**32]
        for _ in range(10):
            hi0, lo0 = product(w[0], 0xD2511F53)
            hi1, lo1 = product(w[2], 0xCD9E8D57)
            w = [hi1 ^ w[1] ^ key[0], lo1, hi0 ^ w[3] ^ key[1], lo0]
            key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
        b = min(n, a + 4 * count)
        drop = (torch.stack(w, 1).reshape(-1)[: b - a].double() / 2**32) < round(c["p"] * 2**32) / 2**32
        kept = (~drop).double() / (1 - c["p"])
        out[a:b] = s["res"][a:b].double() + kept * s["x"][a:b].double()
        dx[a:b] = kept * s["dout"][a:b].double()
    return {"out": out, "dx": dx}


def _exact_gn(c, s, segs):
    C, G, nt, B = c["channels"], c["groups"], len(segs) // c["B"], c["B"]
    y, stats = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda"), torch.empty((2, nt, B, G), dtype=torch.float64, device="cuda")
    dx, dgamma, dbeta = torch.empty_like(y), torch.zeros(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    gamma, beta = s["gamma"].double(), s["beta"].double()
    for t, b, rows in segs:
        x = s["x"][rows].double().reshape(-1, G, C // G)
        mu, var = x.mean((0, 2)), x.var((0, 2), correction=0)
        r = (var + 1e-5) ** -0.5
        stats[0, t, b], stats[1, t, b] = mu, r
        h = ((x - mu[:, None]) * r[:, None]).reshape(-1, C)
        z = h * gamma + beta
        y[rows] = z * torch.sigmoid(z)
        if c["train"]:
            u = torch.sigmoid(z)
            d = s["dy"][rows].double() * (u + z * u * (1 - u))
            dgamma += (d * h).sum(0)
            dbeta += d.sum(0)
            e, hg = (d * gamma).reshape(-1, G, C // G), h.reshape(-1, G, C // G)
            dx[rows] = (r[:, None] * (e - e.mean((0, 2))[:, None] - hg * (e * hg).mean((0, 2))[:, None])).reshape(-1, C)
    got = {"y": y, "mean": stats[0], "rstd": stats[1]}
    return got | ({"dx": dx, "dgamma": dgamma, "dbeta": dbeta} if c["train"] else {})


def _exact_xattn(c, s, segs):
    B, S, H, K, D = c["B"], c["keys"], c["heads"], c["kv_heads"], c["dim"]
    R, f64 = s["q"].shape[0], dict(dtype=torch.float64, device="cuda")
    out, lse, dq = torch.zeros((R, H, D), **f64), torch.full((R, H), -math.inf, **f64), torch.zeros((R, H, D), **f64)
    dk, dv = torch.zeros((B, S, K, D), **f64), torch.zeros((B, S, K, D), **f64)
    for t, b, rows in segs:
        keys = torch.arange(S, device="cuda")
        if s["mask"] is not None:
            keys = (s["mask"][t, b] if s["mask"].dim() == 3 else s["mask"][b]).nonzero()[:, 0]
        if not len(keys):
            continue
        most = max(1, int(1e9 // (len(keys) * (H // K))))
        for j in range(K):
            hs = slice(j * (H // K), (j + 1) * (H // K))
            k, v = s["k"][b, keys, j].double(), s["v"][b, keys, j].double()
            for a in range(rows.start, rows.stop, most):
                i = slice(a, min(rows.stop, a + most))
                q = s["q"][i, hs].double()
                w = q @ k.T / math.sqrt(D)
                lse[i, hs] = torch.logsumexp(w, -1)
                w = torch.softmax(w, -1)
                out[i, hs] = w @ v
                if c["train"]:
                    g = s["dout"][i, hs].double()
                    dv[b, keys, j] += torch.einsum("rhk,rhd->kd", w, g)
                    w = w * (g @ v.T - (g * out[i, hs]).sum(-1, keepdim=True)) / math.sqrt(D)
                    dq[i, hs] = w @ k
                    dk[b, keys, j] += torch.einsum("rhk,rhd->kd", w, q)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if c["train"] else out
