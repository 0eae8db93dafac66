"""tdp_cross_attn and tdp_cross_attn_grad against the plain 64-bit form, at the lengths, heads, strides and masks where they
can go wrong."""
import math

import numpy as np
import pytest

import block_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


RAGGED = (2, (5, 9, 14), (2, 2, 2), (2, 3, 3))
FLAT = (1, (3, 8, 12), (1, 2, 2), (0, 2, 2))


def one(T, B=1):
    return (B, (1, 1, T), (1, 1, 1), (0, 0, 0))


def _mask(kind, nt, B, S, rng):
    if kind == "none":
        return None
    if kind == "tile":                       # random states, some tiles keeping none
        m = rng.random((nt, B, S)) < 0.4
        m[rng.random((nt, B)) < 0.3] = False
        return m
    m = np.zeros((B, S), bool)
    for b in range(B):
        n = [S, S // 2, 1, 0][b % 4] if kind != "empty" else 0
        m[b, :n] = True
        if kind == "left":
            m[b] = m[b, ::-1].copy()
        if kind == "holes":
            m[b] = rng.random(S) < 0.5
            if S > 200:
                m[b, 60:200] = False
    return m


def run(tdp, geom, dtype, H, K, D, S, kind, grad, layout="plain", scale=None, seed=0, amp=1.0, dirty=True, stream=None):
    import torch
    B, dims, tiles, overlap = geom
    rng = np.random.default_rng(seed)
    segs, R = ref.segments(B, dims, tiles, overlap)
    nt = len(segs) // B
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    t = lambda *s: (torch.from_numpy(rng.standard_normal(s, dtype=np.float32)) * amp).to(dt).cuda()  # noqa: E731
    if layout == "fused":                    # one projection's output: slices with wider rows
        qkv = t(R, H + 3, D)
        q = qkv[:, 2:2 + H]
        kv = t(B, S, 2, K, D)
        k, v = kv[:, :, 0], kv[:, :, 1]
    elif layout == "heads":                  # head-major rows and states
        q = t(H, R, D).transpose(0, 1)
        k, v = t(B, K, S, D).transpose(1, 2), t(K, B, S, D).permute(1, 2, 0, 3)
    elif layout == "shared":                 # one item's states broadcast to all items
        q, k, v = t(R, H, D), t(1, S, K, D).expand(B, S, K, D), t(1, S, K, D).expand(B, S, K, D)
    else:
        q, k, v = t(R, H, D), t(B, S, K, D), t(B, S, K, D)
    mask = _mask(kind, nt, B, S, rng)
    host = [x.float().cpu().numpy().astype(np.float64) for x in (q, k, v)]
    if mask is not None and dirty and layout != "shared":     # what no mask keeps is not defined
        gone = torch.from_numpy(~mask.reshape(-1, B, S).any(0)).cuda()
        k[gone], v[gone] = float("nan"), float("inf")
    dout = t(R, H, D) if grad else None
    sc = 1 / math.sqrt(D) if scale is None else scale
    want, smax = ref.xattn(segs, *host, mask, sc, None if dout is None else dout.float().cpu().numpy().astype(np.float64))
    plan = tdp.tdp_plan_create(B, *dims, 8, dtype, tiles, overlap)
    md = None if mask is None else torch.from_numpy(mask).cuda()
    out = torch.full((R, H, D), float("nan"), dtype=dt, device="cuda")
    lse = torch.full((R, H), float("nan"), device="cuda")
    got = {"out": out, "lse": lse}
    torch.cuda.synchronize()
    tdp.tdp_cross_attn(plan, q, k, v, md, out, lse, scale=scale, stream=stream)
    if grad:
        got |= {"dq": torch.full_like(out, float("nan")),
                "dk": torch.full((B, S, K, D), float("nan"), dtype=dt, device="cuda"),
                "dv": torch.full((B, S, K, D), float("nan"), dtype=dt, device="cuda")}
        tdp.tdp_cross_attn_grad(plan, q, k, v, md, out, lse, dout, got["dq"], got["dk"], got["dv"], scale=scale, stream=stream)
    torch.cuda.synchronize()
    unit = ref.xattn_unit(dtype, D, smax)
    for name, x in got.items():
        val, mag = want[name]
        x = x.float().cpu().numpy().astype(np.float64)
        u = ref.xattn_unit("f32", D, smax) if name == "lse" else unit
        inf = np.isinf(val)
        assert np.array_equal(x[inf], val[inf]), f"{name}: rows that keep nothing"
        err = np.abs(x[~inf] - val[~inf])
        bad = ~(err <= u * mag[~inf] + 1e-30)
        assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / (u * mag[~inf] + 1e-30)):.3g} of the bound, nan {np.isnan(err).sum()}"
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,H,K", [(64, 4, 4), (128, 4, 2), (40, 3, 1), (8, 2, 2), (80, 6, 6), (128, 8, 1), (104, 2, 1)])
@pytest.mark.parametrize("grad", [False, True])
def test_head_layouts(tdp, dtype, D, H, K, grad):
    run(tdp, FLAT, dtype, H, K, D, 150, "none", grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [1, 2, 63, 64, 65, 127, 128, 129, 255, 257, 640, 1000])
def test_lengths_of_the_states(tdp, dtype, S):
    run(tdp, FLAT, dtype, 2, 1, 64, S, "none", True)
    run(tdp, RAGGED, dtype, 2, 2, 128, S, "left", True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 513])
def test_lengths_of_the_rows(tdp, dtype, T):
    run(tdp, one(T), dtype, 2, 2, 64, 200, "none", True)
    run(tdp, one(T, B=3), dtype, 4, 1, 128, 130, "length", True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["length", "left", "holes", "tile", "empty"])
@pytest.mark.parametrize("geom", [FLAT, RAGGED, (5, (2, 3, 7), (1, 1, 2), (0, 0, 1))], ids=["one item", "ragged", "five items"])
def test_masks(tdp, dtype, kind, geom):
    run(tdp, geom, dtype, 4, 2, 64, 333, kind, True)
    run(tdp, geom, dtype, 2, 2, 128, 90, kind, True, seed=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["fused", "heads", "shared"])
def test_strides(tdp, dtype, layout):
    run(tdp, RAGGED, dtype, 4, 2, 80, 140, "holes", True, layout)
    run(tdp, one(5, B=2), dtype, 4, 4, 128, 700, "length", True, layout)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,K,S", [(1, 8, 2, 5000), (1, 4, 4, 3000), (3, 32, 2, 4097), (1, 16, 1, 20000)])
@pytest.mark.parametrize("kind", ["none", "length", "holes"])
def test_few_rows_long_states(tdp, dtype, T, H, K, S, kind):
    """The states split over blocks and joined."""
    run(tdp, one(T, B=2), dtype, H, K, 128, S, kind, False)
    run(tdp, one(T, B=4), dtype, H, K, 64, S, kind, False, seed=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_scores(tdp, dtype):
    """Scores of some hundreds: the running maximum grows by more than an exponential can hold."""
    run(tdp, FLAT, dtype, 2, 2, 64, 500, "none", True, scale=4.0, amp=3.0)
    run(tdp, one(2), dtype, 2, 2, 64, 4000, "none", False, scale=4.0, amp=3.0)
    run(tdp, FLAT, dtype, 2, 2, 64, 300, "none", True, scale=-1.0)
    run(tdp, FLAT, dtype, 2, 2, 64, 300, "none", True, scale=0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(tdp, dtype):
    """More row blocks than the device holds at a time, in more than one state tile and head."""
    run(tdp, (1, (8, 32, 48), (1, 2, 2), (0, 4, 4)), dtype, 4, 2, 64, 200, "holes", True)
    run(tdp, (3, (4, 30, 41), (2, 3, 2), (1, 2, 5)), dtype, 2, 2, 128, 260, "tile", True)


def test_no_states(tdp):
    import torch
    plan = tdp.tdp_plan_create(2, 1, 1, 5, 8, "bf16", (1, 1, 1), (0, 0, 0))
    q = torch.randn(10, 2, 64, device="cuda").bfloat16()
    k = torch.empty(2, 0, 2, 64, device="cuda", dtype=torch.bfloat16)
    out, lse, dq = torch.ones_like(q), torch.ones(10, 2, device="cuda"), torch.ones_like(q)
    tdp.tdp_cross_attn(plan, q, k, k, None, out, lse)
    tdp.tdp_cross_attn_grad(plan, q, k, k, None, out, lse, torch.ones_like(q), dq, torch.empty_like(k), torch.empty_like(k))
    assert (out == 0).all() and (lse == -math.inf).all() and (dq == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_every_time(tdp, dtype):
    import torch
    first = run(tdp, RAGGED, dtype, 4, 2, 64, 333, "tile", True)
    for _ in range(3):
        again = run(tdp, RAGGED, dtype, 4, 2, 64, 333, "tile", True)
        assert all(torch.equal(first[n].view(torch.uint8), again[n].view(torch.uint8)) for n in first)


def test_another_stream(tdp):
    import torch
    s = torch.cuda.Stream()
    run(tdp, one(2, B=2), "bf16", 4, 2, 128, 3000, "length", False, stream=s)
    run(tdp, RAGGED, "f32", 4, 2, 64, 200, "tile", True, stream=s)
    run(tdp, RAGGED, "bf16", 4, 2, 64, 200, "tile", True, stream=s.cuda_stream)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_in_a_graph(tdp, dtype):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    plan = tdp.tdp_plan_create(2, 2, 6, 9, 8, dtype, (1, 2, 1), (0, 1, 0))
    R = 2 * plan.total_tile_tokens
    q, k, v, dout = (torch.randn(*s, device="cuda").to(dt) for s in ((R, 4, 64), (2, 150, 2, 64), (2, 150, 2, 64), (R, 4, 64)))
    bufs = lambda: [torch.zeros_like(q), torch.zeros(R, 4, device="cuda"), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]  # noqa: E731
    ws = torch.empty(max(1, tdp.tdp_cross_attn_workspace(plan, q, k, v, grad=True),
                         tdp.tdp_cross_attn_workspace(plan, q, k, v)), dtype=torch.uint8, device="cuda")

    def step(b):
        tdp.tdp_cross_attn(plan, q, k, v, None, b[0], b[1], ws=ws)
        tdp.tdp_cross_attn_grad(plan, q, k, v, None, b[0], b[1], dout, b[2], b[3], b[4], ws=ws)
    a, b = bufs(), bufs()
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for new in range(2):
        if new:
            q.normal_()
            step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradient_against_differences(tdp):
    """fp32: dL along random directions, L = sum(w * out), against central differences of the operator itself.  A step of
    2^-7 leaves a third-derivative term of 1e-4 and a rounding of 1e-6 / 2^-7 of |L|'s terms."""
    import torch
    rng = np.random.default_rng(5)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).cuda()  # noqa: E731
    plan = tdp.tdp_plan_create(2, 2, 5, 7, 8, "f32", (1, 2, 1), (0, 1, 0))
    R, H, K, D, S = 2 * plan.total_tile_tokens, 4, 2, 32, 70
    x = {"q": t(R, H, D), "k": t(2, S, K, D), "v": t(2, S, K, D)}
    w = t(R, H, D)
    mask = torch.from_numpy(rng.random((plan.n_tiles, 2, S)) < 0.6).cuda()
    out, lse = torch.empty_like(w), torch.empty(R, H, device="cuda")

    def loss(y):
        tdp.tdp_cross_attn(plan, y["q"], y["k"], y["v"], mask, out, lse)
        return float((out.double() * w.double()).sum())
    loss(x)
    d = {n: torch.empty_like(y) for n, y in x.items()}
    tdp.tdp_cross_attn_grad(plan, x["q"], x["k"], x["v"], mask, out, lse, w, d["q"], d["k"], d["v"])
    for n in x:
        u, h = t(*x[n].shape), 2.0 ** -7
        fd = (loss({**x, n: x[n] + h * u}) - loss({**x, n: x[n] - h * u})) / (2 * h)
        an = float((d[n].double() * u.double()).sum())
        terms = float((d[n].double() * u.double()).abs().sum())
        assert abs(fd - an) <= 2e-3 * terms + 1e-3, n


def test_offsets_past_32_bits(tdp):
    """States that lie past 2^31 elements: only the last item's last ones are kept."""
    import torch
    B, S, K, D = 5, 1 << 20, 4, 128
    assert B * S * K * D > 1 << 31
    plan = tdp.tdp_plan_create(B, 1, 1, 1, 8, "bf16", (1, 1, 1), (0, 0, 0))
    k = torch.zeros(B, S, K, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(B, S, K, D, dtype=torch.bfloat16, device="cuda")
    n = 100
    k[-1, -n:], v[-1, -n:] = torch.randn(n, K, D, device="cuda").bfloat16(), torch.randn(n, K, D, device="cuda").bfloat16()
    mask = torch.zeros(B, S, dtype=torch.uint8, device="cuda")
    mask[-1, -n:] = 1
    q = torch.randn(B, 8, D, device="cuda").bfloat16()
    out = torch.empty_like(q)
    tdp.tdp_cross_attn(plan, q, k, v, mask, out)
    assert (out[:-1] == 0).all()
    want, smax = ref.xattn([(0, 0, 0, 1)], *(x.float().cpu().numpy().astype(np.float64) for x in (q[-1:], k[-1:, -n:], v[-1:, -n:])), None, D ** -0.5)
    err = np.abs(out[-1].float().cpu().numpy() - want["out"][0][0])
    assert (err <= ref.xattn_unit("bf16", D, smax) * want["out"][1][0]).all()


@pytest.mark.parametrize("S", [2, 4, 9, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_few_states_lose_no_digits(tdp, S, D):
    """With few states dP and delta nearly cancel.  dS and the gradient are each rounded to bf16 once: a rounding's error
    is uniform over half a spacing, at most 2^-8 / sqrt(3) in the mean square, and two of them are independent."""
    import torch
    geom = B, dims, tiles, overlap = FLAT
    segs, R = ref.segments(B, dims, tiles, overlap)
    rng = np.random.default_rng(S)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).bfloat16().cuda()  # noqa: E731
    H, K = 8, 4
    q, k, v, dout = t(R, H, D), t(B, S, K, D), t(B, S, K, D), t(R, H, D)
    want, _ = ref.xattn(segs, *(x.double().cpu().numpy() for x in (q, k, v)), None, 1 / math.sqrt(D), dout.double().cpu().numpy())
    plan = tdp.tdp_plan_create(B, *dims, 8, "bf16", tiles, overlap)
    out, lse, dq, dk, dv = torch.empty_like(q), torch.empty((R, H), device="cuda"), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    tdp.tdp_cross_attn(plan, q, k, v, None, out, lse)
    tdp.tdp_cross_attn_grad(plan, q, k, v, None, out, lse, dout, dq, dk, dv)
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        val = want[name][0]
        err = np.linalg.norm(x.double().cpu().numpy() - val) / np.linalg.norm(val)
        assert err < math.sqrt(2) * 2.0**-8 / math.sqrt(3), (name, err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "holes", "length"])
def test_gradients_of_few_rows_long_states(tdp, dtype, kind):
    """dq's sums over the states, split over blocks (fp32) and joined."""
    run(tdp, one(64), dtype, 4, 4, 128, 2900, kind, True)
    run(tdp, one(3, B=2), dtype, 6, 2, 64, 1300, kind, True, seed=4)
