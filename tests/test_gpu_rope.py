"""tdp_rope and its gradient against 64-bit angles."""
import numpy as np
import pytest

import block_ref
import linear_ref as ref

pytestmark = pytest.mark.gpu
U = ref.U32


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


GEOMETRY = {"ragged": (2, (3, 7, 10), (1, 2, 2), (0, 1, 2)), "tokens": (5, (1, 1, 1), (1, 1, 1), (0, 0, 0)),
            "frames": (1, (9, 4, 5), (3, 1, 2), (2, 0, 1)), "line": (2, (1, 1, 300), (1, 1, 1), (0, 0, 0))}


def _make(tdp, geometry, dtype, far=1 << 10, seed=0):
    B, dims, tiles, overlap = GEOMETRY[geometry]
    segs, R = block_ref.segments(B, dims, tiles, overlap)
    plan = tdp.tdp_plan_create(B, *dims, 8, dtype, tiles, overlap)
    r = np.random.default_rng(seed)
    Q = np.empty(6 * R, np.int32)
    for _, _, r0, T in segs:
        start = r.integers(-far, far, (3, T))
        Q[6 * r0:6 * (r0 + T)] = np.stack([start, start + r.integers(1, 40, (3, T))], -1).reshape(-1)
    return plan, segs, R, Q


def _tolerance(size, want, scale, dtype):
    """cos and sin are off by 2^-24 of a half turn (the angle's rounding, pi 2^-24), two units of 2^-24 of their own (sincospi)
    and one for the scale; two products and a sum.  bf16 takes the fast functions: off by 2^-21.19 within half a turn, 7 units, and
    the angle is rounded once more."""
    units = np.pi + 2 + 1 + 3 if dtype == "f32" else 2 * np.pi + 7 + 1 + 3
    return units * U * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0) + 1e-37


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("geometry", GEOMETRY)
@pytest.mark.parametrize("heads,dim,rot", [(1, 64, 64), (3, 128, 128), (5, 80, 48), (17, 40, 40), (2, 32, 2), (40, 128, 64), (1, 8, 6), (2, 256, 254)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_turns(tdp, dtype, geometry, heads, dim, rot, layout):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    plan, segs, R, Q = _make(tdp, geometry, dtype)
    r = np.random.default_rng(1)
    freq, axis = 10000.0 ** -r.random(rot // 2), r.integers(0, 3, rot // 2)
    table = tdp.tdp_rope_table(freq, axis).cuda()
    x = torch.from_numpy(r.standard_normal((R, heads, dim))).to(dt).cuda()
    Qd, at, scale = torch.from_numpy(Q).cuda(), ("middle", "start")[heads % 2], 1.25 if dim == 80 else 1.0
    _, angle = ref.angles(segs, Q, freq, axis, at == "middle")
    out = torch.full((R * heads * dim + 64,), 3.0, dtype=dt, device="cuda")
    for back, f in ((False, tdp.tdp_rope), (True, tdp.tdp_rope_grad)):
        view = out[:-64].view(R, heads, dim)
        f(plan, x, Qd, table, view, layout=layout, at=at, scale=scale)
        want, size = ref.turn(x.double().cpu().numpy(), angle, scale, layout == "interleaved", back)
        got = view.double().cpu().numpy()
        assert (np.abs(got - want) <= _tolerance(size, want, scale, dtype))[..., :rot].all()
        assert torch.equal(view[..., rot:], x[..., rot:]) and (out[-64:] == 3).all()
        y = x.clone()                      # in place
        f(plan, y, Qd, table, y, layout=layout, at=at, scale=scale)
        assert torch.equal(y, view)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_a_projection(tdp, dtype):
    """Queries and keys turned where they lie, beside values that stay; and heads in front of rows."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    plan, segs, R, Q = _make(tdp, "ragged", dtype)
    Qd, table = torch.from_numpy(Q).cuda(), tdp.tdp_rope_table(*tdp.tdp_rope_freqs((12, 10, 10))[:2]).cuda()
    qkv = torch.randn(R, 6, 64, device="cuda").to(dt)
    want = torch.empty(R, 4, 64, dtype=dt, device="cuda")
    tdp.tdp_rope(plan, qkv[:, :4].contiguous(), Qd, table, want)
    kept = qkv[:, 4:].clone()
    front = torch.empty(4, R, 64, dtype=dt, device="cuda")
    tdp.tdp_rope(plan, qkv[:, :4], Qd, table, front.transpose(0, 1))
    tdp.tdp_rope(plan, qkv[:, :4], Qd, table, qkv[:, :4])
    assert torch.equal(qkv[:, :4], want) and torch.equal(qkv[:, 4:], kept) and torch.equal(front.transpose(0, 1), want)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 50])
def test_far_positions(tdp, far):
    """Angles of positions to the ends of int32, at frequencies whose product with them 64-bit floats hold to 2^-20 turns; the
    reference multiplies in whole numbers."""
    import torch
    plan, segs, R, Q = _make(tdp, "line", "f32", far)
    freq = np.array([1.0, 0.1, 1e-3, 3.7e-6, 2.0 ** -20, 311.0])
    axis = np.array([0, 1, 2, 0, 1, 2])
    turn64 = [int(f * 2 ** 80 / (4 * np.pi)) for f in freq]      # off by 2^-53 of itself: 2^-20 turns at 2^32 and the frequencies to 1
    x = torch.ones(R, 1, 12, device="cuda")
    out = torch.empty_like(x)
    tdp.tdp_rope(plan, x, torch.from_numpy(Q).cuda(), tdp.tdp_rope_table(freq, axis).cuda(), out)
    pos2 = np.concatenate([Q[6 * r0:6 * (r0 + T)].reshape(3, T, 2).astype(object).sum(-1).T for _, _, r0, T in segs])
    got = out[:, 0].double().cpu().numpy()
    for i, f in enumerate(freq):
        turns = np.array([float((int(p) * turn64[i]) % 2 ** 80) / 2.0 ** 80 for p in pos2[:, axis[i]]])
        c, s = np.cos(2 * np.pi * turns), np.sin(2 * np.pi * turns)
        tol = 2 * (np.pi + 6) * U + 2 * np.pi * max(f, 1e-9) * 2 * far * 2.0 ** -53 * 2
        assert (np.abs(got[:, i] - (c - s)) < tol).all() and (np.abs(got[:, i + 6] - (s + c)) < tol).all()


def test_gradient_is_the_transpose(tdp):
    """sum(turned(x) g) = sum(x turned back(g)), and both against differences: the operator is linear."""
    import torch
    plan, segs, R, Q = _make(tdp, "frames", "f32")
    freq, axis, scale = tdp.tdp_rope_freqs((8, 8, 8), scaling="yarn", factor=4.0, length=512.0)
    Qd, table = torch.from_numpy(Q).cuda(), tdp.tdp_rope_table(freq, axis).cuda()
    x, g, d = (torch.randn(R, 3, 56, device="cuda") for _ in range(3))
    y, dx, y2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    tdp.tdp_rope(plan, x, Qd, table, y, scale=scale)
    tdp.tdp_rope(plan, x + d, Qd, table, y2, scale=scale)
    tdp.tdp_rope_grad(plan, g, Qd, table, dx, scale=scale)
    dot = lambda a, b: (float((a.double() * b.double()).sum()), float((a.double() * b.double()).abs().sum()))  # noqa: E731
    (a, s), (b, _) = dot(y, g), dot(x, dx)
    assert abs(a - b) < 16 * U * s * 2
    (a, s), (b, t) = dot(y2.double() - y.double(), g), dot(d, dx)
    assert abs(a - b) < 64 * U * (s + t)


def test_split_positions(tdp):
    """Positions as tdp_split leaves them, normalised or not: scores of queries and keys turned by the same shift agree."""
    import torch
    import workloads as wk
    wl = wk.by_name("tiny")
    plan = tdp.tdp_plan_create(wl.B, wl.F, wl.H, wl.W, wl.C, wl.dtype, wl.num_tiles, wl.overlap)
    X, P, _ = wk.make_inputs(wl)
    Xd, Pd = torch.from_numpy(X).cuda(), torch.from_numpy(P).cuda()
    Y, Q, mn, mx = tdp.alloc_split_outputs(plan, "cuda")
    tdp.tdp_pos_bounds(plan, Pd, mn, mx)
    table = tdp.tdp_rope_table(*tdp.tdp_rope_freqs((6, 5, 5))[:2]).cuda()
    x = torch.randn(plan.B * plan.total_tile_tokens, 2, 32, device="cuda")
    got = []
    for normalize in (0, 1):
        tdp.tdp_split(plan, Xd, Pd, mn, normalize, Y, Q)
        out = torch.empty_like(x)
        tdp.tdp_rope(plan, x, Q, table, out)
        got.append([torch.einsum("thd,shd->hts", out[a:b], out[a:b]) for a, b in zip(plan.offsets[:-1], plan.offsets[1:])])
    for a, b in zip(*got):
        assert float((a - b).abs().max()) < 64 * 2.0 ** -20 * float(a.abs().max())


def test_captured(tdp):
    import torch
    plan, segs, R, Q = _make(tdp, "ragged", "bf16")
    Qd, table = torch.from_numpy(Q).cuda(), tdp.tdp_rope_table(*tdp.tdp_rope_freqs((32, 0, 0))[:2]).cuda()
    x = torch.randn(R, 4, 64, device="cuda").bfloat16()
    want, out = torch.empty_like(x), torch.empty_like(x)
    tdp.tdp_rope(plan, x, Qd, table, want, layout="interleaved")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tdp.tdp_rope(plan, x, Qd, table, out, layout="interleaved")
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_elements_past_32_bits(tdp):
    import torch
    n = (1 << 18) + 5
    plan = tdp.tdp_plan_create(1, 1, 1, n, 8, "bf16", (1, 1, 1), (0, 0, 0))
    x = torch.empty(n, 64, 256, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, 64, 256, device="cuda").bfloat16()
    Q = torch.arange(3 * n * 2, dtype=torch.int32, device="cuda")
    few = tdp.tdp_plan_create(1, 1, 1, 3, 8, "bf16", (1, 1, 1), (0, 0, 0))
    table = tdp.tdp_rope_table(*tdp.tdp_rope_freqs((64, 32, 32))[:2]).cuda()
    want = torch.empty(3, 64, 256, dtype=torch.bfloat16, device="cuda")
    tdp.tdp_rope(few, x[-3:].clone(), Q.view(3, n, 2)[:, -3:].contiguous(), table, want)
    tdp.tdp_rope(plan, x, Q, table, x)
    assert torch.equal(x[-3:], want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_sines_of_every_angle(tdp, layout):
    """fp32: an angle is taken to its nearest quarter turn and a remainder of at most an eighth, which 24 bits hold to 2^-28 turns (and
    2^-32 for the last bits of 64 that are left out); the sines then are a unit of 2^-23 off and no more, small ones too."""
    import torch
    plan, segs, R, Q = _make(tdp, "line", "f32", 1 << 12, seed=5)
    r = np.random.default_rng(6)
    n = 120
    freq, axis = np.pi * (1 + r.integers(0, 64, n) / 32) * (1 + 2.0 ** -r.uniform(8, 24, n)), r.integers(0, 3, n)       # next to parts of a turn
    freq[::3] = r.random(n // 3)
    x = torch.zeros(R, 1, 2 * n, device="cuda")
    (x[..., 0::2] if layout == "interleaved" else x[..., :n]).fill_(1)
    Qd, table = torch.from_numpy(Q).cuda(), tdp.tdp_rope_table(freq, axis).cuda()
    _, angle = ref.angles(segs, Q, freq, axis, True)
    for f, sign in ((tdp.tdp_rope, 1), (tdp.tdp_rope_grad, -1)):
        out = torch.empty_like(x)
        f(plan, x, Qd, table, out, layout=layout)
        got = out[:, 0].double().cpu().numpy()
        c, s = (got[:, 0::2], got[:, 1::2]) if layout == "interleaved" else (got[:, :n], got[:, n:])
        # angles of 64 bits are 2^-53 of themselves off, twice, up to 2^12 * 10
        turn = 2 * np.pi * (2.0 ** -28 + 2.0 ** -32) + 4 * np.abs(angle) * 2.0 ** -53
        for v, want, slope in ((c, np.cos(angle), np.sin(angle)), (s, sign * np.sin(angle), np.cos(angle))):
            assert (np.abs(v - want) <= turn * (np.abs(slope) + turn) + 2.0 ** -23 * np.abs(want) + 1e-12).all()


def test_scale_is_read_in_every_call(tdp):
    """A factor that a program keeps in a tensor and changes there."""
    import torch
    plan, segs, R, Q = _make(tdp, "frames", "f32")
    Qd, table = torch.from_numpy(Q).cuda(), tdp.tdp_rope_table(*tdp.tdp_rope_freqs((8, 8, 8))[:2]).cuda()
    x = torch.randn(R, 2, 48, device="cuda")
    one, two, want = (torch.empty_like(x) for _ in range(3))
    for scale in (torch.tensor(1.0), np.array(1.0, np.float32)):
        tdp.tdp_rope(plan, x, Qd, table, one, scale=scale)
        scale += 1
        tdp.tdp_rope(plan, x, Qd, table, two, scale=scale)
        tdp.tdp_rope(plan, x, Qd, table, want, scale=2.0)
        assert torch.equal(two, want) and not torch.equal(one, two)
