"""tdp_group_norm and tdp_group_norm_grad against the plain 64-bit form."""
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
TINY = (1, (3, 8, 12), (1, 2, 2), (0, 2, 2))
LONG = (1, (6, 40, 50), (1, 1, 2), (0, 0, 3))


def run(tdp, geom, dtype, C, G, act, grad, affine=True, level=0.5, size=1.0, eps=1e-5, seed=0, inplace=False, stream=None):
    import torch
    B, dims, tiles, overlap = geom
    rng = np.random.default_rng(seed)
    segs, R = ref.segments(B, dims, tiles, overlap)
    nt = len(segs) // B
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    t = lambda a: torch.from_numpy(np.asarray(a, np.float32)).to(dt).cuda()  # noqa: E731
    h = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    x = t(rng.standard_normal((R, C)) * size * (0.5 + rng.random(C)) + level * rng.standard_normal(C))
    gamma, beta = (t(1 + 0.3 * rng.standard_normal(C)), t(0.3 * rng.standard_normal(C))) if affine else (None, None)
    dy = t(rng.standard_normal((R, C))) if grad else None
    want = ref.gnorm(segs, nt, B, h(x), G, h(gamma) if affine else np.ones(C), h(beta) if affine else np.zeros(C), eps,
                     act == "silu", None if dy is None else h(dy))
    plan = tdp.tdp_plan_create(B, *dims, 8, dtype, tiles, overlap)
    f = dict(device="cuda", dtype=torch.float32)
    nan = lambda *s: torch.full(s, float("nan"), **f)  # noqa: E731
    y = x.clone() if inplace else nan(R, C).to(dt)
    got = {"y": y, "mean": nan(nt, B, G), "rstd": nan(nt, B, G)}
    torch.cuda.synchronize()
    tdp.tdp_group_norm(plan, y if inplace else x, G, gamma, beta, y, got["mean"], got["rstd"], eps=eps, act=act, stream=stream)
    if grad:
        got |= {"dx": dy.clone() if inplace else nan(R, C).to(dt), "dgamma": nan(C), "dbeta": nan(C)}
        if inplace:
            torch.cuda.synchronize()
        tdp.tdp_group_norm_grad(plan, x, G, gamma, beta, got["mean"], got["rstd"], got["dx"] if inplace else dy, got["dx"],
                                got["dgamma"], got["dbeta"], act=act, stream=stream)
    torch.cuda.synchronize()
    for name, v in got.items():
        val, mag = want[name]
        v = h(v)
        # fp32: sums of a few hundred values a thread, joined over threads and blocks: 2^-24 * 64 of the
        # terms' magnitudes; bf16 results are rounded once, 2^-8 of the value
        tol = 64 * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(val) if v.ndim == 2 and dtype == "bf16" else 0) + 1e-30
        bad = ~(np.abs(v - val) <= tol)
        assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(v - val) / tol):.3g} of the bound"
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("C,G", [(16, 4), (128, 32), (120, 20), (64, 1), (64, 64), (24, 8), (8, 1), (520, 13), (2056, 4)])
def test_channels_and_groups(tdp, dtype, act, C, G):
    run(tdp, TINY, dtype, C, G, act, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("geom", [RAGGED, LONG, (3, (1, 1, 7), (1, 1, 1), (0, 0, 0)), (2, (1, 16, 16), (1, 1, 1), (0, 0, 0)),
                                  (1, (1, 1, 257), (1, 1, 1), (0, 0, 0)), (1, (4, 30, 41), (2, 3, 2), (1, 2, 5))],
                         ids=["ragged", "long", "seven", "256", "257", "tiles"])
@pytest.mark.parametrize("affine", [True, False])
def test_lengths(tdp, dtype, geom, affine):
    run(tdp, geom, dtype, 48, 6, "silu", True, affine)
    run(tdp, geom, dtype, 256, 32, "none", True, affine, seed=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_token(tdp, dtype):
    run(tdp, (3, (1, 1, 1), (1, 1, 1), (0, 0, 0)), dtype, 64, 2, "silu", True)
    got = run(tdp, (2, (1, 1, 1), (1, 1, 1), (0, 0, 0)), dtype, 8, 8, "none", False, affine=False)
    assert (got["y"] == 0).all()          # a group of one value


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mean_far_from_zero(tdp, dtype):
    """A level some thousand times the spread: squares of the values themselves would leave nothing of the variance."""
    run(tdp, LONG, dtype, 32, 4, "none", True, level=0.0, size=1.0)
    import torch
    rng = np.random.default_rng(2)
    segs, R = ref.segments(*LONG)
    x = rng.standard_normal((R, 32)) + 3000.0
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    xt = torch.from_numpy(x).to(dt).cuda()
    plan = tdp.tdp_plan_create(LONG[0], *LONG[1], 8, dtype, LONG[2], LONG[3])
    nt = len(segs)
    mean, rstd = torch.empty(nt, 1, 4, device="cuda"), torch.empty(nt, 1, 4, device="cuda")
    tdp.tdp_group_norm(plan, xt, 4, None, None, torch.empty_like(xt), mean, rstd)
    want = ref.gnorm(segs, nt, 1, xt.double().cpu().numpy(), 4, np.ones(32), np.zeros(32), 1e-5, False)
    # squared deviations are summed about values of the data: the spread's own size, 2^-24 * 64
    assert np.abs(rstd.cpu().numpy() / want["rstd"][0] - 1).max() < 2e-5
    assert np.abs(mean.cpu().numpy() / want["mean"][0] - 1).max() < 2e-6


def test_constant_input(tdp):
    import torch
    plan = tdp.tdp_plan_create(1, 4, 20, 20, 8, "f32", (1, 2, 2), (0, 2, 2))
    x = torch.full((plan.total_tile_tokens, 32), 7.25, device="cuda")
    mean, rstd, y = torch.empty(4, 1, 8, device="cuda"), torch.empty(4, 1, 8, device="cuda"), torch.empty_like(x)
    tdp.tdp_group_norm(plan, x, 8, None, None, y, mean, rstd, eps=1e-5)
    assert (mean == 7.25).all() and (y == 0).all() and torch.allclose(rstd, torch.tensor(1e-5 ** -0.5, device="cuda"), rtol=1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_streams(tdp, dtype):
    import torch
    run(tdp, RAGGED, dtype, 64, 8, "silu", True, inplace=True)
    run(tdp, LONG, dtype, 64, 8, "silu", True, inplace=True)
    run(tdp, RAGGED, dtype, 64, 8, "silu", True, stream=torch.cuda.Stream())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_every_time(tdp, dtype):
    import torch
    a = run(tdp, LONG, dtype, 64, 8, "silu", True)
    for _ in range(3):
        b = run(tdp, LONG, dtype, 64, 8, "silu", True)
        assert all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in a)


def test_captured_in_a_graph(tdp):
    import torch
    plan = tdp.tdp_plan_create(1, 4, 20, 20, 8, "bf16", (1, 2, 2), (0, 2, 2))
    x, dy = (torch.randn(plan.total_tile_tokens, 64, device="cuda").bfloat16() for _ in range(2))
    ws = torch.empty(tdp.tdp_group_norm_workspace(plan, 64, 8), dtype=torch.uint8, device="cuda")
    bufs = lambda: [torch.zeros_like(x), torch.zeros(4, 1, 8, device="cuda"), torch.zeros(4, 1, 8, device="cuda"),  # noqa: E731
                    torch.zeros_like(x), torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")]

    def step(b):
        tdp.tdp_group_norm(plan, x, 8, None, None, b[0], b[1], b[2], act="silu", ws=ws)
        tdp.tdp_group_norm_grad(plan, x, 8, None, None, b[1], b[2], dy, b[3], b[4], b[5], act="silu", ws=ws)
    a, b = bufs(), bufs()
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for new in range(2):
        if new:
            x.normal_()
            step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_gradient_against_differences(tdp):
    """fp32, L = sum(w * y), central differences with a step of 2^-7 of values of order one."""
    import torch
    rng = np.random.default_rng(5)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).cuda()  # noqa: E731
    plan = tdp.tdp_plan_create(2, 2, 5, 7, 8, "f32", (1, 2, 1), (0, 1, 0))
    R, C, G, n = 2 * plan.total_tile_tokens, 32, 4, plan.n_tiles
    v = {"x": t(R, C), "gamma": t(C) + 1, "beta": t(C)}
    w, y, mean, rstd = t(R, C), torch.empty(R, C, device="cuda"), torch.empty(n, 2, G, device="cuda"), torch.empty(n, 2, G, device="cuda")

    def loss(u):
        tdp.tdp_group_norm(plan, u["x"], G, u["gamma"], u["beta"], y, mean, rstd, act="silu")
        return float((y.double() * w.double()).sum())
    loss(v)
    d = {k: torch.empty_like(a) for k, a in v.items()}
    tdp.tdp_group_norm_grad(plan, v["x"], G, v["gamma"], v["beta"], mean, rstd, w, d["x"], d["gamma"], d["beta"], act="silu")
    for k in v:
        u, step = t(*v[k].shape), 2.0 ** -7
        fd = (loss({**v, k: v[k] + step * u}) - loss({**v, k: v[k] - step * u})) / (2 * step)
        prod = d[k].double() * u.double()
        assert abs(fd - float(prod.sum())) <= 2e-3 * float(prod.abs().sum()) + 1e-3, k


def test_offsets_past_32_bits(tdp):
    """The last tile's rows lie past 2^31 elements."""
    import torch
    plan = tdp.tdp_plan_create(1, 64, 512, 520, 8, "bf16", (4, 2, 2), (0, 0, 0))
    C, G, n = 128, 4, plan.n_tiles
    R = plan.total_tile_tokens
    assert R * C > 1 << 31
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda").normal_()
    y, mean, rstd = torch.empty_like(x), torch.empty(n, 1, G, device="cuda"), torch.empty(n, 1, G, device="cuda")
    tdp.tdp_group_norm(plan, x, G, None, None, y, mean, rstd)
    a = int(plan.offsets[-2])
    last = x[a:].double().reshape(-1, G, C // G)
    mu, var = last.mean((0, 2)), last.var((0, 2), correction=0)
    assert (mean[-1, 0].double() - mu).abs().max() < 1e-6 and (rstd[-1, 0].double() * (var + 1e-5).sqrt() - 1).abs().max() < 1e-5
    want = ((last - mu[:, None]) / (var + 1e-5).sqrt()[:, None]).reshape(-1, C)
    assert ((y[a:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all()
    dx = y                                      # the gradient of sum(x_hat * dy) written over y
    tdp.tdp_group_norm_grad(plan, x, G, None, None, mean, rstd, x, dx)
    # dy = x: dx = rstd * (x - mean(x) - h * mean(x h)) = h * (1 - (1 - eps rstd^2)): nearly zero everywhere
    assert dx[a:].float().abs().max() < 1e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,G", [(1280, 32), (2080, 2080), (3000, 25), (4096, 1), (5000, 5)])
def test_rows_wider_than_a_block(tdp, dtype, C, G):
    """Several slabs of whole groups a row, the last one narrower; groups wider than a block."""
    run(tdp, TINY, dtype, C, G, "silu", True)
    run(tdp, (2, (2, 17, 23), (1, 2, 2), (0, 2, 2)), dtype, C, G, "none", True)
