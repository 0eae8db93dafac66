"""Cases for the operators around a per-tile transformer block's projections: norm, rotary positions, products in 8 bits.

  norm    root-mean-square norm of rows with the residual's addition; forward in the plan's type or in 8 bits (e4m3, a scale a
          row), forward and gradients; the normalised rows kept in 8 bits, and the gradients from them
  rope    rotation of the tiles' heads by the positions that the split hands out (forward; gradient)
  linear  product of 8-bit rows and 8-bit weights with a scale a row and a channel, bias and residual; from rows that are
          in 8 bits already, or that are brought there first

`run` computes a case in its plain form (elementary torch operations in 32 bits, angles in 64, rounded once at the end),
or, where `own` is true, through the package's entry points.  `exact` is the definition in 64 bits; of an output in 8 bits
it is the value before that rounding.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}
E4M3 = torch.float8_e4m3fn
MOST8 = 448.0                   # e4m3's largest value
LEAST = 2.0 ** -100             # magnitude below which a row's scale falls no further
EPS = 1e-6


# ---------------------------------------------------------------- cases
def _plan(B, F, H, W, nf=1, nh=1, nw=1, of=0, oh=0, ow=0):
    return dict(B=B, F=F, H=H, W=W, nf=nf, nh=nh, nw=nw, of=of, oh=oh, ow=ow)


TINY = _plan(1, 3, 8, 12, 1, 2, 2, 0, 2, 2)            # the repository's workloads
SMALL = _plan(1, 16, 32, 48, 1, 2, 2, 0, 8, 8)
MEDIUM = _plan(1, 16, 64, 96, 1, 4, 4, 0, 8, 8)
TEMPORAL = _plan(2, 32, 68, 120, 2, 3, 3, 4, 8, 8)
RAGGED = _plan(2, 9, 17, 30, 2, 2, 2, 2, 4, 4)         # odd extents: tiles of many sizes
TOKEN = _plan(8, 1, 1, 1)                              # one token per item


def _norm(name, dtype, rows, channels, form, res):
    """form: "y" (the plan's type), "y8" (8 bits), "train" (forward and gradients), "keep8" (training's forward, the normalised
    rows kept in 8 bits), "grad8" (the gradients from such rows)."""
    return dict(name=name, op="norm", dtype=dtype, rows=rows, channels=channels, form=form, res=res)


def _rope(name, plan, dtype, heads, dim, rot, layout, axes, scaling, far, train, fused):
    return dict(name=name, op="rope", dtype=dtype, heads=heads, dim=dim, rot=rot, layout=layout, axes=axes, scaling=scaling,
                far=far, train=train, fused=fused, **plan)


def _linear(name, dtype, rows, inner, outer, quant, bias, res):
    return dict(name=name, op="linear", dtype=dtype, rows=rows, inner=inner, outer=outer, quant=quant, bias=bias, res=res)


def listed():
    return [
        # one token of eight items between two sublayers, on its way to an 8-bit projection: latency counts
        _norm("norm token 8-bit", "bf16", 8, 4096, "y8", True),
        # every tile row of the medium latent on its way to an 8-bit projection: serving
        _norm("norm medium 8-bit", "bf16", 168960, 2048, "y8", True),
        # the small latent's rows in training, the stream kept for the gradient
        _norm("norm train", "bf16", 35840, 2048, "train", True),
        # gradients from rows that were kept in 8 bits; an odd number of rows and of vectors a row
        _norm("norm grad from 8 bits", "f32", 5381, 1000, "grad8", True),
        # eight items' single tokens far into a stream, frequencies scaled for it: a decoding step
        _rope("rope token", TOKEN, "bf16", 40, 128, 128, "half", 1, "yarn", True, False, True),
        # queries and keys of the medium latent's tiles, slices of a fused projection
        _rope("rope medium", MEDIUM, "bf16", 32, 128, 128, "interleaved", 3, "none", False, False, True),
        # training on tiles of many sizes, part of the head
        _rope("rope train part", RAGGED, "f32", 6, 80, 48, "half", 3, "ntk", False, True, False),
        # the temporal tile set, narrow heads, forward and gradient
        _rope("rope train temporal", TEMPORAL, "bf16", 8, 64, 64, "half", 3, "none", False, True, False),
        # one token of eight items through a projection: bound by the weights' bytes
        _linear("linear token", "bf16", 8, 4096, 4096, False, False, False),
        # the small latent's rows through an odd-sized projection in fp32
        _linear("linear odd f32", "f32", 1237, 1040, 1004, True, True, False),
        # the small latent's attention outputs, brought to 8 bits, through the output projection onto the residual
        _linear("linear small out", "bf16", 35840, 2048, 2048, True, True, True),
        # the medium latent's rows through a fused query, key and value projection: the largest
        _linear("linear medium", "bf16", 168960, 2048, 4096, False, False, False),
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
    p = _plan(rng.choice([1, 1, 2, 8]), f[0], h[0], w[0], f[1], h[1], w[1], f[2], h[2], w[2])
    return p if _geometry(p)[3] * p["B"] <= cells else _draw_plan(rng, cells)


def draw(rng):
    op = rng.choice(["norm", "rope", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    unit = 16 // ESIZE[dtype]
    if op == "norm":
        C = unit * _loguniform(rng, 1, 1024)
        rows = _loguniform(rng, 1, min(200_000, 300_000_000 // C))
        form = rng.choice(["y", "y8", "train", "keep8", "grad8"])
        return dict(op=op, dtype=dtype, rows=max(1, rows // 2) if form == "train" else rows, channels=C, form=form,
                    res=rng.random() < 0.6)
    if op == "rope":
        dim = rng.choice([32, 40, 64, 64, 80, 96, 128, 128])
        heads = rng.choice([1, 2, 6, 8, 16, 24, 40])
        rot = dim if rng.random() < 0.6 else 2 * unit * rng.randint(1, dim // (2 * unit))
        train = rng.random() < 0.4
        return dict(op=op, dtype=dtype, heads=heads, dim=dim, rot=rot, layout=rng.choice(["half", "interleaved"]), axes=rng.choice([1, 3, 3]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), far=rng.random() < 0.3, train=train, fused=rng.random() < 0.5,
                    **_draw_plan(rng, 300_000_000 // (heads * dim * (2 if train else 1))))
    rows = _loguniform(rng, 1, 170_000)
    inner = 16 * _loguniform(rng, 2, 512)
    outer = unit * _loguniform(rng, 4, 8192 // unit)
    while rows * inner * outer > 1.2e12 or rows * outer > 7e8:
        rows = (rows + 1) // 2
    return dict(op=op, dtype=dtype, rows=rows, inner=inner, outer=outer, quant=rng.random() < 0.5, bias=rng.random() < 0.5,
                res=rng.random() < 0.4)


# ---------------------------------------------------------------- geometry
def _boxes(L, n, o):
    i = np.arange(n)
    o = o if n > 1 else 0
    lo = np.where(i > 0, i * L // n - o // 2, 0)
    hi = np.where(i < n - 1, (i + 1) * L // n + o - o // 2, L)
    return lo, hi - lo


def _geometry(c):
    """Tokens per tile [nt], token offset per tile [nt], tile of each token [tot], tokens in all."""
    s = [_boxes(c["F"], c["nf"], c["of"])[1], _boxes(c["H"], c["nh"], c["oh"])[1], _boxes(c["W"], c["nw"], c["ow"])[1]]
    T = (s[0][:, None, None] * s[1][None, :, None] * s[2][None, None, :]).reshape(-1).astype(np.int64)
    off = np.cumsum(T) - T
    return T, off, np.repeat(np.arange(len(T)), T), int(T.sum())


def _positions(c, seed):
    """Tile-major positions as the split leaves them, int32 [B * tot * 6], and for every row the place of its first
    start there and the step from one axis to the next."""
    T, off, tile, tot = _geometry(c)
    lo, size = zip(*(_boxes(c[k], c["n" + k.lower()], c["o" + k.lower()]) for k in "FHW"))
    iF, iH, iW = tile // (c["nh"] * c["nw"]), tile // c["nw"] % c["nh"], tile % c["nw"]
    j = np.arange(tot) - off[tile]
    w, h, f = j % size[2][iW], j // size[2][iW] % size[1][iH], j // (size[2][iW] * size[1][iH])
    step = (8, 32, 32)                                          # a latent cell in frames and pixels
    r = np.random.default_rng(seed)
    cell = np.stack([f + lo[0][iF], h + lo[1][iH], w + lo[2][iW]], 0)          # [3, tot]
    first = r.integers(0, 1 << 20 if c["far"] else 64, (c["B"], 3))
    b = np.arange(c["B"])[:, None]
    rows = c["B"] * off[tile] + b * T[tile] + j                 # [B, tot]
    at = 6 * c["B"] * off[tile] + 6 * b * T[tile] + 2 * j
    Q = np.empty(6 * c["B"] * tot, np.int32)
    place, axis = np.empty(c["B"] * tot, np.int64), np.empty(c["B"] * tot, np.int64)
    for d in range(3):
        start = cell[d] * step[d] + first[:, d:d + 1]
        Q[at + 2 * d * T[tile]] = start
        Q[at + 2 * d * T[tile] + 1] = start + step[d]
    place[rows], axis[rows] = at, np.broadcast_to(2 * T[tile], rows.shape)
    return Q, place, axis


# ---------------------------------------------------------------- rotary frequencies
BASE, FACTOR, LENGTH = 10000.0, 8.0, 8192.0


def _pairs(c):
    n = c["rot"] // 2
    return (n, 0, 0) if c["axes"] == 1 else (n - 2 * (n // 3), n // 3, n // 3)


def _freqs(c):
    """Frequency and axis of every pair, and the factor of cos and sin."""
    f, axis = [], []
    for a, n in enumerate(_pairs(c)):
        base = BASE * FACTOR ** (n / (n - 1)) if c["scaling"] == "ntk" and n > 1 else BASE
        f += [base ** (-i / n) for i in range(n)]
        axis += [a] * n
    f = np.array(f)
    if c["scaling"] == "linear":
        f = f / FACTOR
    if c["scaling"] == "yarn":
        keep = np.clip((LENGTH * f / (2 * math.pi) - 1) / (32 - 1), 0, 1)      # turns within the trained length: 1 to 32
        f = f * keep + f / FACTOR * (1 - keep)
    return f, np.array(axis), 0.1 * math.log(FACTOR) + 1 if c["scaling"] == "yarn" else 1.0


# ---------------------------------------------------------------- inputs
def _to8(x):
    """x [R, C] in e4m3 with a scale a row, largest magnitude / 448: values and scales."""
    top = x.abs().amax(-1, keepdim=True).clamp_min(LEAST)
    # 448 x / top: values midway between two of e4m3's come out exact, and no product overflows
    return ((0.875 * x) / (top / 512)).clamp(-MOST8, MOST8).to(E4M3), top[:, 0] / MOST8


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)

    def like(*shape, kind=dt):
        return torch.empty(shape, dtype=kind, device="cuda")

    s = {"case": case}
    if case["op"] == "norm":
        R, C, form = case["rows"], case["channels"], case["form"]
        # a residual stream: some channels far larger than the rest
        size = torch.exp(torch.randn((C,), generator=g, device="cuda") * 0.7)
        x = torch.randn((R, C), generator=g, device="cuda") * size
        s["w"] = normal(C, std=0.2, mean=1.0)
        if form == "grad8":         # what the forward kept
            s["rstd"] = 1 / torch.sqrt(x.square().mean(-1) + EPS)
            s["x8"], s["x8_scale"] = _to8(x * s["rstd"][:, None])
        else:
            s |= {"x": x.to(dt), "res": (torch.randn((R, C), generator=g, device="cuda") * size * 3).to(dt) if case["res"] else None}
        if form in ("train", "grad8"):
            s |= {"dy": normal(R, C, std=0.01), "dh": normal(R, C, std=0.01) if case["res"] else None}
        if own:
            f32 = torch.float32
            s |= {"plan": _own_plan(dict(TINY, dtype=case["dtype"]))}
            if form != "grad8":
                s |= {"h": like(R, C) if case["res"] else None, "y": None if form == "y8" else like(R, C)}
            if form in ("train", "keep8"):
                s["rstd"] = like(R, kind=f32)
            if form in ("y8", "keep8"):
                s |= {"v8": like(R, C, kind=E4M3), "scale": like(R, kind=f32)}
            if form in ("train", "grad8"):
                s |= {"dx": like(R, C), "dw": like(C, kind=f32)}
        return s
    if case["op"] == "rope":
        Q, place, axis = _positions(case, seed)
        R, H, D = len(place), case["heads"], case["dim"]
        s["x"] = normal(R, H + 8, D)[:, :H] if case["fused"] else normal(R, H, D)       # the values lie behind, as a projection writes them
        s |= {"Q": torch.from_numpy(Q).cuda(), "place": torch.from_numpy(place).cuda(), "step": torch.from_numpy(axis).cuda()}
        if case["train"]:
            s["dout"] = normal(R, H, D, std=0.01)
        freq, axis, s["scale"] = _freqs(case)
        s |= {"freq": torch.from_numpy(freq).cuda(), "axis": torch.from_numpy(axis).cuda()}
        if own:
            import blend_tdp_tile_gb300 as tdp
            freq, axis, scale = tdp.tdp_rope_freqs(_pairs(case), BASE, case["scaling"], FACTOR, LENGTH)
            s |= {"plan": _own_plan(case), "table": tdp.tdp_rope_table(freq, axis).cuda(), "scale": scale,
                  "out": like(R, H, D), "dx": like(R, H, D) if case["train"] else None}
        return s
    R, K, N = case["rows"], case["inner"], case["outer"]
    w = torch.randn((N, K), generator=g, device="cuda") * torch.exp(torch.randn((N, 1), generator=g, device="cuda") * 0.3) / math.sqrt(K)
    s["w8"], s["ws"] = _to8(w)
    x = torch.randn((R, K), generator=g, device="cuda") * torch.exp(torch.randn((R, 1), generator=g, device="cuda"))
    if case["quant"]:
        s["x"] = x.to(dt)
    else:
        s["x8"], s["xs"] = _to8(x)
    s |= {"bias": normal(N, std=0.1) if case["bias"] else None, "res": normal(R, N) if case["res"] else None}
    if own:
        s |= {"plan": _own_plan(dict(TINY, dtype=case["dtype"])), "out": like(R, N)}
        if case["quant"]:
            s |= {"x8": like(R, K, kind=E4M3), "xs": like(R, kind=torch.float32)}
    return s


def _own_plan(c):
    import blend_tdp_tile_gb300 as tdp
    return tdp.tdp_plan_create(c["B"], c["F"], c["H"], c["W"], 8, c["dtype"],
                               (c["nf"], c["nh"], c["nw"]), (c["of"], c["oh"], c["ow"]))


# ---------------------------------------------------------------- one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_norm(s):
    import blend_tdp_tile_gb300 as tdp
    form = s["case"]["form"]
    if form == "grad8":
        tdp.tdp_rms_norm_grad(s["plan"], s["dy"], s["dx"], s["w"], s["rstd"], x8=s["x8"], x8_scale=s["x8_scale"], dh=s["dh"], dw=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    r = {"h": s["h"]} if s["case"]["res"] else {}
    if form == "y":
        tdp.tdp_rms_norm(s["plan"], s["x"], s["w"], s["y"], res=s["res"], h=s["h"], eps=EPS)
        return r | {"y": s["y"]}
    if form == "y8":
        tdp.tdp_rms_norm(s["plan"], s["x"], s["w"], None, res=s["res"], h=s["h"], y8=s["v8"], y8_scale=s["scale"], eps=EPS)
        return r | {"y8": s["v8"], "y8_scale": s["scale"]}
    r |= {"y": s["y"], "rstd": s["rstd"]}
    if form == "keep8":
        tdp.tdp_rms_norm(s["plan"], s["x"], s["w"], s["y"], res=s["res"], h=s["h"], rstd=s["rstd"], x8=s["v8"], x8_scale=s["scale"], eps=EPS)
        return r | {"x8": s["v8"], "x8_scale": s["scale"]}
    tdp.tdp_rms_norm(s["plan"], s["x"], s["w"], s["y"], res=s["res"], h=s["h"], rstd=s["rstd"], eps=EPS)
    h = s["h"] if s["case"]["res"] else s["x"]          # without a residual the rows themselves are the stream
    tdp.tdp_rms_norm_grad(s["plan"], s["dy"], s["dx"], s["w"], s["rstd"], h=h, dh=s["dh"], dw=s["dw"])
    return r | {"dx": s["dx"], "dw": s["dw"]}


def _own_rope(s):
    import blend_tdp_tile_gb300 as tdp
    tdp.tdp_rope(s["plan"], s["x"], s["Q"], s["table"], s["out"], layout=s["case"]["layout"], scale=s["scale"])
    if not s["case"]["train"]:
        return s["out"]
    tdp.tdp_rope_grad(s["plan"], s["dout"], s["Q"], s["table"], s["dx"], layout=s["case"]["layout"], scale=s["scale"])
    return {"out": s["out"], "dx": s["dx"]}


def _own_linear(s):
    import blend_tdp_tile_gb300 as tdp
    if s["case"]["quant"]:
        tdp.tdp_quant8(s["plan"], s["x"], s["x8"], s["xs"])
    tdp.tdp_matmul8(s["plan"], s["x8"], s["xs"], s["w8"], s["ws"], s["out"], bias=s["bias"], res=s["res"])
    return {"out": s["out"], "x8": s["x8"], "x8_scale": s["xs"]} if s["case"]["quant"] else s["out"]


def _plain_norm(s):
    form, dt, w = s["case"]["form"], DTYPES[s["case"]["dtype"]], s["w"].float()
    r = {}
    if form == "grad8":
        rstd, u = s["rstd"][:, None], s["x8"].float() * s["x8_scale"][:, None]
    else:
        h = (s["x"].float() + s["res"].float()).to(dt) if s["case"]["res"] else s["x"]
        if s["case"]["res"]:
            r["h"] = h
        u = h.float()
        rstd = 1 / torch.sqrt(u.square().mean(-1, keepdim=True) + EPS)
        u = u * rstd
        if form == "y8":
            r["y8"], r["y8_scale"] = _to8(u * w)
            return r
        r["y"] = (u * w).to(dt)
        if form == "y":
            return r
        r["rstd"] = rstd[:, 0]
        if form == "keep8":
            r["x8"], r["x8_scale"] = _to8(u)
            return r
    dy = s["dy"].float()
    r["dw"] = (dy * u).sum(0)
    dy = dy * w
    dx = (dy - u * (dy * u).mean(-1, keepdim=True)) * rstd
    r["dx"] = (dx + s["dh"].float() if s["case"]["res"] else dx).to(dt)
    return r


def _plain_rope(s):
    c = s["case"]
    rot, interleaved = c["rot"], c["layout"] == "interleaved"
    start = s["Q"][s["place"][:, None] + s["step"][:, None] * s["axis"]]               # [R, pairs]
    end = s["Q"][s["place"][:, None] + s["step"][:, None] * s["axis"] + 1]
    angle = (start.double() + end.double()) / 2 * s["freq"]
    cos, sin = ((f(angle) * s["scale"]).float()[:, None] for f in (torch.cos, torch.sin))

    def turned(x, sin):
        y = x.float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
        a, b = a * cos - b * sin, a * sin + b * cos
        y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
        return torch.cat((y.to(x.dtype), x[..., rot:]), -1)

    out = turned(s["x"], sin)
    return {"out": out, "dx": turned(s["dout"], -sin)} if c["train"] else out


def _plain_linear(s):
    c = s["case"]
    x8, xs = _to8(s["x"].float()) if c["quant"] else (s["x8"], s["xs"])
    out = x8.float() @ s["w8"].float().t()
    out = out * xs[:, None] * s["ws"]
    if c["bias"]:
        out = out + s["bias"].float()
    if c["res"]:
        out = out + s["res"].float()
    out = out.to(DTYPES[c["dtype"]])
    return {"out": out, "x8": x8, "x8_scale": xs} if c["quant"] else out


_plain = {"norm": _plain_norm, "rope": _plain_rope, "linear": _plain_linear}
_own = {"norm": _own_norm, "rope": _own_rope, "linear": _own_linear}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = ESIZE[case["dtype"]]
    if case["op"] == "norm":
        R, C, form = case["rows"], case["channels"], case["form"]
        n, more = R * C, 2 if case["res"] else 0
        b = e * n * (1 + more) + e * C if form != "grad8" else e * C + 4 * R       # x, res -> h
        b += n + 4 * R if form in ("y8", "keep8", "grad8") else 0                   # -> y8 or x8; or from x8
        b += e * n if form not in ("y8", "grad8") else 0                            # -> y
        b += 4 * R if form in ("train", "keep8") else 0                             # -> rstd
        b += e * n * (2 + more // 2) + 4 * C if form in ("train", "grad8") else 0   # dy, dh -> dx, dw
        return {"bytes": b, "flops": n * {"y": 6, "y8": 9, "train": 16, "keep8": 9, "grad8": 12}[form]}
    if case["op"] == "rope":
        rows = case["B"] * _geometry(case)[3]
        n, t = rows * case["heads"] * case["dim"], 2 if case["train"] else 1
        return {"bytes": t * 2 * e * n + 24 * rows, "flops": t * 3 * rows * case["heads"] * case["rot"]}
    R, K, N = case["rows"], case["inner"], case["outer"]
    b = N * K + 4 * N + R * K + 4 * R + e * R * N * (2 if case["res"] else 1) + (e * N if case["bias"] else 0)
    return {"bytes": b + (e * R * K if case["quant"] else 0), "flops": 2 * R * K * N + (4 * R * K if case["quant"] else 0)}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "linear": _exact_linear}[case["op"]](case, s)


def _exact_8(x):
    """The values that are rounded to e4m3, and the rows' scales."""
    most = torch.maximum(x.abs().max(1).values, torch.tensor(LEAST, dtype=torch.float64, device="cuda"))
    return x * MOST8 / most[:, None], most / MOST8


def _exact_grid(v):
    """The e4m3 value next to v, ties to an even last digit; |v| <= 448: four digits above 2^-6, steps of 2^-9 below."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_norm(c, s):
    C, form, dt, w = c["channels"], c["form"], DTYPES[c["dtype"]], s["w"].double()
    got = {}
    if form == "grad8":
        rstd, unit = s["rstd"].double(), s["x8"].double() * s["x8_scale"].double()[:, None]
    else:
        kept = s["x"].double()
        if c["res"]:
            got["h"] = kept = kept + s["res"].double()
        stream = kept.to(dt).double()                           # the norm is of the stream as it is kept
        rstd = (torch.einsum("rc,rc->r", stream, stream) / C + EPS) ** -0.5
        unit = stream * rstd[:, None]
        if form == "y8":
            got["y8"], got["y8_scale"] = _exact_8(unit * w)
            return got
        got["y"] = unit * w
        if form == "y":
            return got
        got["rstd"] = rstd
        if form == "keep8":
            got["x8"], got["x8_scale"] = _exact_8(unit)
            return got
    dy = s["dy"].double()
    got["dw"] = torch.einsum("rc,rc->c", dy, unit)
    dot = torch.einsum("rc,rc,c->r", dy, unit, w) / C
    got["dx"] = torch.addcmul(dy * w, unit, dot[:, None], value=-1) * rstd[:, None]
    if c["res"]:
        got["dx"] += s["dh"]
    return got


def _exact_rope(c, s):
    H, D, rot = c["heads"], c["dim"], c["rot"]
    freq, axis, scale = _freqs(c)
    Q, place, step = (s[k].cpu().numpy() for k in ("Q", "place", "step"))
    pos = [(Q[place + d * step].astype(np.float64) + Q[place + d * step + 1]) / 2 for d in range(3)]
    first, second = (np.arange(rot // 2) * 2, np.arange(rot // 2) * 2 + 1) if c["layout"] == "interleaved" else \
        (np.arange(rot // 2), np.arange(rot // 2) + rot // 2)

    def turned(x, sign):
        y = x.double()
        for i in range(rot // 2):
            angle = torch.from_numpy(pos[axis[i]]).cuda() * freq[i]
            turn = torch.polar(torch.full_like(angle, scale), sign * angle)[:, None]
            z = turn * torch.complex(x[:, :, first[i]].double(), x[:, :, second[i]].double())
            y[:, :, first[i]], y[:, :, second[i]] = z.real, z.imag
        return y

    out = turned(s["x"], 1)
    return {"out": out, "dx": turned(s["dout"], -1)} if c["train"] else out


def _exact_linear(c, s):
    R, N = c["rows"], c["outer"]
    got = {}
    if c["quant"]:
        got["x8"], got["x8_scale"] = _exact_8(s["x"].double())
        x, xs = _exact_grid(got["x8"]), got["x8_scale"]
    else:
        x, xs = s["x8"].double(), s["xs"].double()
    w = s["w8"].double() * s["ws"].double()[:, None]
    out = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    if c["bias"]:
        out += s["bias"].double()
    if c["res"]:
        out += s["res"].double()
    out.addmm_(x * xs[:, None], w.T)
    return got | {"out": out} if c["quant"] else out
