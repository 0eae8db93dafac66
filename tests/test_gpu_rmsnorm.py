"""tdp_rms_norm, its gradients and 8-bit rows against 64 bits."""
import numpy as np
import pytest

import linear_ref as ref

pytestmark = pytest.mark.gpu
U = ref.U32


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


def _plan(tdp, dtype):
    return tdp.tdp_plan_create(1, 1, 1, 1, 8, dtype, (1, 1, 1), (0, 0, 0))


def _np(t):
    return t.double().cpu().numpy()


def _guarded(n, kind, fill=3.0):
    """A buffer of n elements with 64 more behind it that a call must leave as they are."""
    import torch
    if kind == torch.uint8:
        return torch.full((n + 64,), 0x55, dtype=kind, device="cuda")
    return torch.full((n + 64,), fill, dtype=kind, device="cuda")


# an element, less and more than a warp, an odd number of vectors, one warp's most, several warps, the longest rows
MANY = [(5000, 24), (3001, 136), (2000, 768), (1300, 1040), (2500, 2048), (700, 2992), (999, 4096), (641, 5120), (330, 8192)]        # rows for every SM
SHAPES = [(1, 8), (5, 16), (131, 24), (67, 136), (33, 1000), (200, 2048), (9, 2056), (1, 4096), (3, 8192)]


def _inputs(rows, C, dt, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + rows * 7 + C)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return (r(rows, C) * torch.exp(r(C))).to(dt), (r(rows, C) * 2).to(dt), (r(C) * 0.3 + 1).to(dt), (r(rows, C) * 0.1).to(dt), (r(rows, C) * 0.1).to(dt)


def _roundings(C):
    """Relative error of rstd in units of 2^-24: a sum of squares has at most 64 terms a lane and 13 joins behind them, each a
    rounding, and so have the squares; half of it reaches rstd, with the mean, eps, root and reciprocal."""
    return (64 + 13 + 1) / 2 + 4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", SHAPES + MANY)
@pytest.mark.parametrize("res,weight", [(True, True), (False, True), (True, False)])
def test_forward(tdp, dtype, rows, C, res, weight):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, s, w, _, _ = _inputs(rows, C, dt)
    s, w = s if res else None, w if weight else None
    n = rows * C
    h, y = _guarded(n, dt), _guarded(n, dt)
    y8, x8 = _guarded(n, torch.uint8), _guarded(n, torch.uint8)
    rstd, ys, xs = (_guarded(rows, torch.float32) for _ in range(3))
    tdp.tdp_rms_norm(_plan(tdp, dtype), x, w, y[:n].view(rows, C), res=s, h=h[:n], rstd=rstd[:rows], y8=y8[:n], y8_scale=ys[:rows],
                     x8=x8[:n], x8_scale=xs[:rows], eps=1e-5)
    for t, k in ((h, n), (y, n), (rstd, rows), (ys, rows), (xs, rows)):
        assert (t[k:] == 3).all()
    assert (y8[n:] == 0x55).all() and (x8[n:] == 0x55).all()
    want_h = (x.float() + s.float()).to(dt) if res else x
    assert torch.equal(h[:n].view(rows, C), want_h)
    rs, u, out = ref.rms_norm(_np(want_h), _np(w) if weight else np.ones(C), 1e-5)
    k = _roundings(C) * U
    assert (np.abs(_np(rstd[:rows]) - rs) <= k * rs).all()
    # two products behind rstd, and the plan's type
    tol = (k + 2 * U) * np.abs(out) + (2.0 ** -8 * np.abs(out) if dtype == "bf16" else 0) + 1e-37
    assert (np.abs(_np(y[:n].view(rows, C)) - out) <= tol).all()
    for v8, scale, v in ((y8, ys, out), (x8, xs, u)):
        _, want = ref.rows8(v)
        got = _np(scale[:rows])
        assert (np.abs(got - want) <= (k + 5 * U) * want).all()     # products, the maximum's and the division's rounding
        val = _np(v8[:n].view(torch.float8_e4m3fn).view(rows, C).float())
        assert (np.abs(val) <= 448).all() and (np.abs(val).max(1) == 448).all()
        # half a step of e4m3 where it lands, and what v and its scale were off before
        off = np.abs(val * got[:, None] - v)
        assert (off <= got[:, None] * ref.half_step8(v / got[:, None]) * (1 + 1e-5) + (2 * k + 12 * U) * np.abs(v)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", SHAPES + MANY + [(70, 4096)])
def test_quant(tdp, dtype, rows, C):
    """To the value: of bf16 rows 448 v / m is a quotient of whole numbers below 2^9 and 2^8 times a power of two, and 2^-17
    away from any tie that it does not meet; of fp32 rows those within 2^-21 of a tie may go either way."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = _inputs(rows, C, dt, 3)[0]
    x8, xs = torch.empty((rows, C), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    tdp.tdp_quant8(_plan(tdp, dtype), x, x8, xs)
    v, scale = ref.rows8(_np(x))
    assert (np.abs(_np(xs) - scale) <= U * scale).all()
    got, want = _np(x8.float()), ref.e4m3(v)
    if dtype == "f32":
        near = ref.e4m3(v * (1 + 2.0 ** -21)) != ref.e4m3(v * (1 - 2.0 ** -21))
        got, want = got[~near], want[~near]
    assert np.array_equal(got, want)


def test_quant_ties(tdp):
    """Every value midway between two of e4m3's, with a largest magnitude that is no power of two."""
    import torch
    for top in (1.0, 1.75, 3.5, 448.0, 1.3125):
        grid = np.unique(ref.e4m3(np.linspace(0, 448, 100001)))
        mid = (grid[1:] + grid[:-1]) / 2 * top / 448
        row = np.concatenate([mid, -mid, [top]])
        row = np.concatenate([row, np.zeros(-len(row) % 8)]).astype(np.float32)
        x = torch.from_numpy(row).cuda()[None].contiguous()
        x8, xs = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(1, device="cuda")
        tdp.tdp_quant8(_plan(tdp, "f32"), x, x8, xs)
        v = row.astype(np.float64) * 448 / top
        exact = (v.astype(np.float32) == v) & ((v * top / 448) == row)
        assert np.array_equal(_np(x8.float())[0][exact], ref.e4m3(v)[exact])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [16, 2048, 4096])
def test_rows_that_hold_anything(tdp, dtype, C):
    """NaN, infinities, zeros, the smallest and the largest values: each row for itself."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.randn(7, C, device="cuda").to(dt)
    x[1, 3], x[2, 5], x[3] = float("nan"), float("-inf"), 0
    x[4] = 0
    x[4, 2] = 2.0 ** -120
    x[5] *= 2.0 ** -60
    plan = _plan(tdp, dtype)
    y, y8, ys = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(7, device="cuda")
    rstd = torch.empty(7, device="cuda")
    tdp.tdp_rms_norm(plan, x, None, y, rstd=rstd, y8=y8, y8_scale=ys, eps=1e-6)
    alone = torch.empty_like(x)
    for i in (0, 5, 6):
        tdp.tdp_rms_norm(plan, x[i:i + 1], None, alone[i:i + 1], eps=1e-6)
        assert torch.equal(alone[i], y[i]) and torch.isfinite(y[i]).all()
    for i in (1, 2):
        assert torch.isnan(ys[i]) and torch.isnan(y8[i].float()).all()
    assert torch.isnan(y[1]).all() and torch.isnan(rstd[1]) and rstd[2] == 0
    assert (y[3] == 0).all() and (y8[3].float() == 0).all() and abs(float(ys[3]) * 448 / 2.0 ** -100 - 1) < 1e-6
    tdp.tdp_rms_norm(plan, x[3:4], None, None, y8=y8[3:4], y8_scale=ys[3:4], eps=1e-20)      # 448 / scale / sqrt(eps) is no float
    assert (y8[3].float() == 0).all()
    # rows of nothing but small values
    v8, vs = torch.empty_like(y8), torch.empty_like(ys)
    tdp.tdp_quant8(plan, x, v8, vs)
    for i in (1, 2):
        assert torch.isnan(vs[i]) and torch.isnan(v8[i].float()).all()
    assert (v8[3:5].float() == 0).all() and torch.isfinite(vs[3:]).all()
    big = torch.full((2, C), torch.finfo(dt).max, dtype=dt, device="cuda")
    big[1, 1:] /= 3
    tdp.tdp_quant8(plan, big, v8[:2], vs[:2])
    assert (v8[0].float() == 448).all() and (v8[1, 1:].float() == 144).all() and v8[1, 0].float() == 448     # 149.3: of 144 and 160


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", SHAPES + [(1500, 64), (700, 2048), (650, 4096), (690, 1040), (700, 2992), (310, 8192)])
@pytest.mark.parametrize("kept", ["h", "x8"])
@pytest.mark.parametrize("dh,weight", [(True, True), (False, False)])
def test_gradients(tdp, dtype, rows, C, kept, dh, weight):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, _, w, dy, back = _inputs(rows, C, dt, 5)
    plan, w, back = _plan(tdp, dtype), w if weight else None, back if dh else None
    rstd, x8, xs = torch.empty(rows, device="cuda"), torch.empty((rows, C), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    tdp.tdp_rms_norm(plan, x, w, None, rstd=rstd, x8=x8, x8_scale=xs)
    n = rows * C
    dx, dw = _guarded(n, dt), _guarded(C, torch.float32)
    saved = dict(h=x) if kept == "h" else dict(x8=x8, x8_scale=xs)
    tdp.tdp_rms_norm_grad(plan, dy, dx[:n].view(rows, C), w, rstd, dh=back, dw=dw[:C], **saved)
    assert (dx[n:] == 3).all() and (dw[C:] == 3).all()
    u = _np(x) * _np(rstd)[:, None] if kept == "h" else _np(x8.float()) * _np(xs)[:, None]
    want, size, want_w, size_w = ref.rms_norm_grad(u, _np(rstd), _np(w) if weight else np.ones(C), _np(dy), _np(back) if dh else np.zeros((rows, C)))
    # the mean has 64 terms a lane and 13 joins, each term three roundings; a few more around it
    tol = (64 + 13 + 3 + 8) * U * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0) + 1e-37
    assert (np.abs(_np(dx[:n].view(rows, C)) - want) <= tol).all()
    # a lane's rows, its block's teams, the blocks' parts: rows in all at most, and no more than that; the terms two roundings
    tol = (min(rows, 700) + 3) * U * size_w
    assert (np.abs(_np(dw[:C]) - want_w) <= tol).all()
    same = torch.empty_like(x)
    tdp.tdp_rms_norm_grad(plan, dy, same, w, rstd, dh=back, **saved)           # without dw
    assert torch.equal(same, dx[:n].view(rows, C))
    for to in ([dy.clone()] if back is None else [dy.clone(), back.clone()]):  # in place
        i = torch.equal(to, dy)
        tdp.tdp_rms_norm_grad(plan, to if i else dy, to, w, rstd, dh=back if i else to, **saved)
        assert torch.equal(to, same)


@pytest.mark.parametrize("res", [False, True])
def test_gradient_against_differences(tdp, res):
    """A step of the inputs along a line moves sum(y gy + h gh), in 64 bits, by the gradient times it; the third derivative
    leaves 1e-7 of it at steps of 1e-4, and fp32 2^-24 * 2^7 of the terms."""
    import torch
    rows, C, eps = 6, 40, 1e-3
    g = torch.Generator().manual_seed(1)
    x, s, dx_, ds_ = (torch.randn(rows, C, generator=g, dtype=torch.float64).float().double() for _ in range(4))
    w, dw_ = (torch.randn(C, generator=g, dtype=torch.float64).float().double() for _ in range(2))
    gy, gh = (torch.randn(rows, C, generator=g, dtype=torch.float64).float().double() for _ in range(2))

    def f(t):
        h = x + t * dx_ + (s + t * ds_ if res else 0)
        return float((gy * torch.from_numpy(ref.rms_norm(h.numpy(), (w + t * dw_).numpy(), eps)[2]) + gh * h).sum())

    c = lambda t: t.float().cuda()  # noqa: E731
    plan, h, rstd = _plan(tdp, "f32"), torch.empty(rows, C, device="cuda"), torch.empty(rows, device="cuda")
    tdp.tdp_rms_norm(plan, c(x), c(w), None, res=c(s) if res else None, h=h, rstd=rstd, eps=eps)
    dx, dw = torch.empty_like(h), torch.empty(C, device="cuda")
    tdp.tdp_rms_norm_grad(plan, c(gy), dx, c(w), rstd, h=h, dh=c(gh), dw=dw)
    terms = dx.double().cpu() * (dx_ + (ds_ if res else 0))
    got = float(terms.sum() + (dw.double().cpu() * dw_).sum())
    size = float(terms.abs().sum() + (dw.double().cpu() * dw_).abs().sum())
    assert abs((f(1e-4) - f(-1e-4)) / 2e-4 - got) < (2.0 ** -17 + 1e-6) * size


def test_in_place_and_nothing(tdp):
    import torch
    plan = _plan(tdp, "bf16")
    x, s, w, dy, _ = _inputs(37, 1024, torch.bfloat16)
    h, y = torch.empty_like(x), torch.empty_like(x)
    tdp.tdp_rms_norm(plan, x, w, y, res=s, h=h)
    a, b = x.clone(), s.clone()
    tdp.tdp_rms_norm(plan, a, w, a, res=b, h=b)         # y over x, h over res
    assert torch.equal(a, y) and torch.equal(b, h)
    none = torch.empty(0, 1024, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((1024,), 5.0, device="cuda")
    tdp.tdp_rms_norm(plan, none, w, none)
    tdp.tdp_quant8(plan, none, none.to(torch.float8_e4m3fn), torch.empty(0, device="cuda"))
    tdp.tdp_rms_norm_grad(plan, none, none, w, torch.empty(0, device="cuda"), h=none, dw=dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("rows,C,dtype", [(400, 16384, "bf16"), (310, 14000, "bf16"), (400, 8192, "f32"), (2, 16384, "bf16")])
def test_longest_rows(tdp, rows, C, dtype):
    """Eight warps a row, eight vectors a lane: the row's result as torch's in 64 bits, forward alone (with and without 8 bits), and
    the gradient's two forms against each other's formula by way of test_gradients' bounds."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, s, w, dy, _ = _inputs(rows, C, dt, 9)
    plan, y, y2, h = _plan(tdp, dtype), torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rstd, y8, ys = torch.empty(rows, device="cuda"), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    tdp.tdp_rms_norm(plan, x, w, y, res=s, h=h, rstd=rstd)
    tdp.tdp_rms_norm(plan, x, w, y2, res=s, y8=y8, y8_scale=ys)
    hd, wd = h.double(), w.double()
    r = (hd.square().mean(1) + 1e-6).rsqrt()
    want = hd * r[:, None] * wd
    k = _roundings(C) * U
    assert ((rstd.double() - r).abs() <= k * r).all()
    tol = (k + 2 * U) * want.abs() + (2.0 ** -8 * want.abs() if dtype == "bf16" else 0) + 1e-37
    assert ((y.double() - want).abs() <= tol).all() and ((y2.double() - want).abs() <= tol).all()
    assert ((y8.double() * ys.double()[:, None] - want).abs() <= ys.double()[:, None] * 2.0 ** -10 + 1.001 * 2.0 ** -4 * want.abs()).all()
    dx, dw = torch.empty_like(x), torch.empty(C, device="cuda")
    tdp.tdp_rms_norm_grad(plan, dy, dx, w, rstd, h=h, dw=dw)
    u = hd * rstd.double()[:, None]
    g = dy.double() * wd
    size = rstd.double()[:, None] * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    want = rstd.double()[:, None] * (g - u * (g * u).mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= 88 * U * size + (2.0 ** -8 * want.abs() if dtype == "bf16" else 0) + 1e-37).all()
    terms = dy.double() * u
    assert ((dw.double() - terms.sum(0)).abs() <= (rows + 3) * U * terms.abs().sum(0)).all()


def test_captured_and_on_streams(tdp):
    """A captured forward and gradient replayed beside the same calls on another stream."""
    import torch
    plan = _plan(tdp, "bf16")
    rows, C = 900, 768
    x, s, w, dy, dh = _inputs(rows, C, torch.bfloat16)
    def buffers():
        e = lambda: torch.empty_like(x)  # noqa: E731
        return dict(y=e(), h=e(), dx=e(), rstd=torch.empty(rows, device="cuda"), dw=torch.empty(C, device="cuda"))
    def call(b):
        tdp.tdp_rms_norm(plan, x, w, b["y"], res=s, h=b["h"], rstd=b["rstd"])
        tdp.tdp_rms_norm_grad(plan, dy, b["dx"], w, b["rstd"], h=b["h"], dh=dh, dw=b["dw"])
    want, a, b = buffers(), buffers(), buffers()
    call(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
    side = torch.cuda.Stream()
    for t in a.values():
        t.fill_(0)
    torch.cuda.synchronize()
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(side):
            call(b)
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(a[k], want[k]) and torch.equal(b[k], want[k]), k


def test_elements_past_32_bits(tdp):
    import torch
    rows, C = (1 << 18) + 3, 16384
    x = torch.empty((rows, C), dtype=torch.bfloat16, device="cuda")
    x[-2:] = torch.randn(2, C, device="cuda").to(torch.bfloat16)
    few = x[-2:].clone()
    plan, v8, vs = _plan(tdp, "bf16"), torch.empty((rows, C), dtype=torch.uint8, device="cuda"), torch.empty(rows, device="cuda")
    w8, ws, y = torch.empty((2, C), dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(few)
    tdp.tdp_rms_norm(plan, few, None, y, y8=w8, y8_scale=ws)
    tdp.tdp_rms_norm(plan, x, None, x, y8=v8, y8_scale=vs)
    assert torch.equal(x[-2:], y) and torch.equal(v8[-2:], w8) and torch.equal(vs[-2:], ws)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(200, 2048), (33, 1000), (2000, 768), (1500, 64), (700, 2992), (400, 8192)])
@pytest.mark.parametrize("res,weight", [(True, True), (False, False)])
def test_norm_rows_in_8_bits_to_the_value(tdp, dtype, rows, C, res, weight):
    """rstd stands in a value and in its row's largest alike: x8 is e4m3 of 448 h / max|h|, y8 of 448 h w / max|h w|, ties to the even one.
    Of bf16 rows h w has 16 digits, and 448 h w / m is 2^-21 away from any tie that it does not meet; of fp32 rows those within 2^-21 of
    a tie (roundings of h w, of the largest and of the quotient: 3 * 2^-24) may go either way."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, s, w, _, _ = _inputs(rows, C, dt, 21)
    s, w = s if res else None, w if weight else None
    x8, y8 = (torch.empty((rows, C), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    xs, ys = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    plan = _plan(tdp, dtype)
    tdp.tdp_rms_norm(plan, x, w, None, res=s, y8=y8, y8_scale=ys, x8=x8, x8_scale=xs)
    h = _np((x.float() + s.float()).to(dt) if res else x)
    for got, v in ((x8, h), (y8, h * (_np(w) if weight else 1.0))):
        got, v = _np(got.float()), ref.rows8(v)[0]
        want = ref.e4m3(v)
        if dtype == "f32":
            near = ref.e4m3(v * (1 + 2.0 ** -21)) != ref.e4m3(v * (1 - 2.0 ** -21))
            got, want = got[~near], want[~near]
        assert np.array_equal(got, want)
    # the same with one of them alone, and beside y
    one, y = torch.empty_like(y8), torch.empty_like(x)
    tdp.tdp_rms_norm(plan, x, w, y, res=s, y8=one, y8_scale=ys)
    assert torch.equal(one.view(torch.uint8), y8.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [1e-6, 1e-30])
def test_norm_rows_of_small_values_in_8_bits(tdp, dtype, eps):
    """Rows of 2^-111 and of 2^-118: at eps = 1e-30 (rstd 1e15) their largest value is above 2^-100 and cancels as it does in other rows, at
    1e-6 (rstd 1000) it counts as 2^-100.  The fp32 value before its rounding to e4m3 is 3 * 2^-24 off, with rstd 2^-22."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    rows, C = 64, 512
    x = _inputs(rows, C, torch.bfloat16, 2)[0].double()
    x /= x.abs().amax(1, keepdim=True)
    x[::2] *= 2.0 ** -111
    x[1::2] *= 2.0 ** -118
    x = x.to(dt)
    x8, xs = torch.empty((rows, C), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    tdp.tdp_rms_norm(_plan(tdp, dtype), x, None, None, x8=x8, x8_scale=xs, eps=eps)
    h = _np(x)
    rstd = float(np.float32(eps)) ** -0.5             # the squares are no floats
    least = np.abs(h).max(1) * rstd < ref.LEAST
    assert least.all() if eps == 1e-6 else not least.any()
    v = h * rstd * 448 / ref.LEAST if eps == 1e-6 else ref.rows8(h * 2.0 ** 100)[0]
    off = np.abs(_np(x8.float()) - v)
    assert (off <= ref.half_step8(v) * (1 + 2.0 ** -18) + np.abs(v) * 2.0 ** -20).all()
    if eps == 1e-30 and dtype == "bf16":
        assert np.array_equal(_np(x8.float()), ref.e4m3(v))
    m = np.maximum(np.abs(h).max(1) * rstd, ref.LEAST)
    assert (np.abs(_np(xs) - m / 448) <= 8 * U * m / 448).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(9, 16), (900, 136), (700, 1040), (400, 8192), (2, 8192)])
@pytest.mark.parametrize("res", [False, True])
def test_smallest_eps_takes_the_same_rows(tdp, dtype, rows, C, res):
    """Below 2^-36 eps has kernels of its own; rstd, of ordinary rows the same to a rounding, stands in no value of 8 bits."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, s, w, _, _ = _inputs(rows, C, dt, 30)
    plan, got = _plan(tdp, dtype), []
    for eps in (2.0 ** -36, 2.0 ** -37, 0.0):
        b = {k: torch.empty((rows, C), dtype=torch.uint8, device="cuda") for k in ("x8", "y8")} | {k: torch.empty(rows, device="cuda") for k in ("x8_scale", "y8_scale", "rstd")}
        h, y = torch.empty_like(x), torch.empty_like(x)
        tdp.tdp_rms_norm(plan, x, w, y, res=s if res else None, h=h, eps=eps, **b)
        got.append(b | {"h": h, "y": y})
    for b in got[1:]:
        assert torch.equal(b["x8"], got[0]["x8"]) and torch.equal(b["y8"], got[0]["y8"]) and torch.equal(b["h"], got[0]["h"])
        for k in ("x8_scale", "y8_scale", "rstd"):
            assert ((b[k] - got[0][k]).abs() <= 8 * U * got[0][k]).all()         # two ways of summing; eps is 2^-37 of it at rstd 1
        assert ((b["y"].double() - got[0]["y"].double()).abs() <= (2 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20) * got[0]["y"].double().abs() + 1e-37).all()


@pytest.mark.parametrize("rows,C", [(3000, 1024), (200, 8192), (40000, 64)])
def test_quant_of_fp32_rows_to_the_value(tdp, rows, C):
    """The fp32 quotient of 0.875 v by m / 512, both rounded as fp32 rounds, and the value next to it: every code, those near a tie too."""
    import torch
    x = _inputs(rows, C, torch.float32, 8)[0]
    x[:, 5::7] = x.abs().amax(1, keepdim=True) * (torch.randint(1, 32, x[:, 5::7].shape, device="cuda").float() / 64)     # next to ties
    x8, xs = torch.empty((rows, C), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    tdp.tdp_quant8(_plan(tdp, "f32"), x, x8, xs)
    v = x.cpu().numpy()
    q = (np.float32(0.875) * v) / (np.abs(v).max(1, keepdims=True) / np.float32(512))
    assert q.dtype == np.float32 and np.array_equal(_np(x8.float()), ref.e4m3(q))
