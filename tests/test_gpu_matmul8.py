"""tdp_matmul8 against 64 bits, and the serving path of the 8-bit operators together."""
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


def _case(rows, K, N, dt, seed=0, whole=False):
    """e4m3 rows and weights with scales, bias, residual.  whole: small integers, whose sums are exact in any order."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + rows + 3 * K + 7 * N)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if whole:
        i = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()  # noqa: E731
        return i(rows, K).to(torch.float8_e4m3fn), torch.ones(rows, device="cuda"), i(N, K).to(torch.float8_e4m3fn), torch.ones(N, device="cuda"), None, None
    return ((r(rows, K) * 60).clamp(-448, 448).to(torch.float8_e4m3fn), torch.exp(r(rows)) * 0.01, (r(N, K) * 60).clamp(-448, 448).to(torch.float8_e4m3fn),
            torch.exp(r(N)) * 0.01, r(N).to(dt), (r(rows, N) * 30).to(dt))


def _check(tdp, dtype, rows, K, N, bias=True, res=True):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x8, xs, w8, ws, b, s = _case(rows, K, N, dt)
    b, s = b if bias else None, s if res else None
    out = torch.full((rows * N + 64,), 3.0, dtype=dt, device="cuda")
    tdp.tdp_matmul8(_plan(tdp, dtype), x8, xs, w8, ws, out[:rows * N], bias=b, res=s)
    assert (out[rows * N:] == 3).all()
    x, w = x8.double() * xs.double()[:, None], w8.double() * ws.double()[:, None]
    want, size = x @ w.T, x.abs() @ w.abs().T
    if bias:
        want, size = want + b.double(), size + b.double().abs()
    if res:
        want, size = want + s.double(), size + s.double().abs()
    # K sums and four more roundings, of terms of any size; truncated sums would be off by a whole step
    tol = 2 * (K + 8) * U * size + (2.0 ** -8 * want.abs() if dtype == "bf16" else 0)
    got = out[:rows * N].view(rows, N).double()
    assert ((got - want).abs() <= tol).all()
    # and over all of them as much as sums of K random roundings are off
    if dtype == "f32" and rows * N > 1000:
        assert float((got - want).norm() / want.norm()) < 2 * (K ** 0.5 + 8) * U


SIZES = [(60000, 64, 8), (30000, 512, 72), (20000, 128, 128), (19000, 256, 384), (300, 96, 8), (70000, 272, 40), (13000, 512, 136), (33, 2048, 2048), (400, 2048, 2048), (1024, 4096, 1024)] + [(1, 16, 8), (8, 4096, 4096), (3, 32, 24), (16, 1040, 136), (17, 128, 128), (40, 48, 1000), (64, 272, 264), (65, 4096, 72), (100, 96, 2048),
         (128, 512, 256), (129, 1040, 1004), (300, 2048, 640), (1237, 1040, 1004), (700, 16, 3000), (4000, 640, 520), (19500, 256, 264),
         (5121, 144, 1000), (10000, 2048, 512)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,K,N", SIZES)
def test_sizes(tdp, dtype, rows, K, N):
    N -= N % (4 if dtype == "f32" else 8)
    _check(tdp, dtype, rows, K, N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias,res", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("rows", [5, 200, 3000])
def test_epilogues(tdp, dtype, bias, res, rows):
    _check(tdp, dtype, rows, 528, 392, bias, res)


@pytest.mark.parametrize("rows,K,N", [(7, 4096, 512), (30, 1024, 256), (100, 2000, 264), (900, 512, 1032), (5000, 1024, 2048), (20000, 256, 512)])
def test_whole_numbers(tdp, rows, K, N):
    """Sums of whole numbers below 2^24 are exact whatever their order: every element equal."""
    import torch
    x8, xs, w8, ws, _, _ = _case(rows, K, N, torch.float32, whole=True)
    out = torch.empty(rows, N, device="cuda")
    tdp.tdp_matmul8(_plan(tdp, "f32"), x8, xs, w8, ws, out)
    assert torch.equal(out.double(), x8.double() @ w8.double().T)


def test_residual_in_place_and_no_rows(tdp):
    import torch
    plan = _plan(tdp, "bf16")
    for rows in (9, 513, 4000):
        x8, xs, w8, ws, b, s = _case(rows, 256, 264, torch.bfloat16)
        out = torch.empty_like(s)
        tdp.tdp_matmul8(plan, x8, xs, w8, ws, out, bias=b, res=s)
        tdp.tdp_matmul8(plan, x8, xs, w8, ws, s, bias=b, res=s)
        assert torch.equal(out, s)
    tdp.tdp_matmul8(plan, x8[:0], xs[:0], w8, ws, s[:0])


@pytest.mark.parametrize("rows", [4, 200, 3000])
def test_rows_of_nan_stay_alone(tdp, rows):
    import torch
    x8, xs, w8, ws, _, _ = _case(rows, 512, 256, torch.float32)
    plan, out, want = _plan(tdp, "f32"), torch.empty(rows, 256, device="cuda"), torch.empty(rows, 256, device="cuda")
    tdp.tdp_matmul8(plan, x8, xs, w8, ws, want)
    x8.view(torch.uint8)[2] = 0x7f
    xs[2] = float("nan")
    tdp.tdp_matmul8(plan, x8, xs, w8, ws, out)
    assert torch.isnan(out[2]).all()
    out[2] = want[2]
    assert torch.equal(out, want)


def test_same_bits_in_a_graph_and_on_streams(tdp):
    import torch
    for rows in (8, 300, 5000):
        x8, xs, w8, ws, b, s = _case(rows, 1024, 768, torch.bfloat16)
        plan = _plan(tdp, "bf16")
        want, a, c = (torch.empty_like(s) for _ in range(3))
        tdp.tdp_matmul8(plan, x8, xs, w8, ws, want, bias=b, res=s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tdp.tdp_matmul8(plan, x8, xs, w8, ws, a, bias=b, res=s)
        side = torch.cuda.Stream()
        for _ in range(20):
            graph.replay()
            with torch.cuda.stream(side):
                tdp.tdp_matmul8(plan, x8, xs, w8, ws, c, bias=b, res=s)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(c, want)


def test_elements_past_32_bits(tdp):
    """Outputs past 2^31: the last rows as in a call of their own."""
    import torch
    rows, K, N = (1 << 17) + 77, 64, 16384
    x8, xs, w8, ws, _, _ = _case(256, K, N, torch.bfloat16)
    x8, xs = x8.view(torch.uint8).repeat(rows // 256 + 1, 1)[:rows].contiguous(), xs.repeat(rows // 256 + 1)[:rows].contiguous()
    plan, out = _plan(tdp, "bf16"), torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    tdp.tdp_matmul8(plan, x8, xs, w8, ws, out)
    want = (x8[-300:].view(torch.float8_e4m3fn).double() * xs[-300:].double()[:, None]) @ (w8.double() * ws.double()[:, None]).T
    assert ((out[-300:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4 * want.abs().max()).all()
    assert torch.equal(out[:256], out[256:512]) and torch.equal(out[rows - 333:rows - 77], out[:256])


def test_block_in_8_bits(tdp):
    """Residual and norm into 8 bits, query projection, rotary positions, attention to conditioning tokens that each tile keeps,
    back to 8 bits, output projection onto the stream: every operator against the formula of its own inputs (tests above);
    here the chain against 64 bits.  Each rounding to e4m3 is off by 2^-4 of its value at most and by 0.027 in the mean square; two of
    them on the way, and bf16's beside them: 0.03 of the attention's share, whose part of the output is its own size."""
    import torch
    torch.manual_seed(2)
    B, dims, tiles, overlap = 2, (3, 8, 12), (1, 2, 2), (0, 2, 2)
    plan = tdp.tdp_plan_create(B, *dims, 8, "bf16", tiles, overlap)
    R, C, H, D, S = B * plan.total_tile_tokens, 256, 4, 64, 40
    bf = dict(dtype=torch.bfloat16, device="cuda")
    cond = tdp.tdp_plan_create(B, 1, 1, S, 8, "bf16", (1, 1, 1), (0, 0, 0))
    P = torch.randint(0, 64, (6 * R,), dtype=torch.int32, device="cuda")
    Pc = torch.randint(0, 64, (B, 3, S, 2), dtype=torch.int32, device="cuda")
    keep = torch.rand(plan.n_tiles, B, S, device="cuda") < 0.5
    keep[0, 1] = False
    x, res, w = torch.randn(R, C, **bf), torch.randn(R, C, **bf), torch.rand(C, **bf) + 0.5
    k, v = torch.randn(B, S, H, D, **bf), torch.randn(B, S, H, D, **bf)
    wq, wo = torch.randn(H * D, C, **bf) / 16, torch.randn(C, H * D, **bf) / 16
    table = tdp.tdp_rope_table(*tdp.tdp_rope_freqs((12, 10, 10))[:2]).cuda()
    e8 = lambda n, c: (torch.empty(n, c, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(n, device="cuda"))  # noqa: E731
    (q8, qs), (o8, os), (h8, hs), (a8, as_) = e8(H * D, C), e8(C, H * D), e8(R, C), e8(R, H * D)
    tdp.tdp_quant8(plan, wq, q8, qs)
    tdp.tdp_quant8(plan, wo, o8, os)
    kr, h, q, out = torch.empty_like(k), torch.empty_like(x), torch.empty(R, H, D, **bf), torch.empty(R, C, **bf)
    tdp.tdp_rope(cond, k.view(B * S, H, D), Pc, table, kr.view(B * S, H, D))
    tdp.tdp_rms_norm(plan, x, w, None, res=res, h=h, y8=h8, y8_scale=hs)
    tdp.tdp_matmul8(plan, h8, hs, q8, qs, q)
    tdp.tdp_rope(plan, q, P, table, q)
    a = torch.empty_like(q)
    tdp.tdp_cross_attn(plan, q, kr, v, keep, a)
    tdp.tdp_quant8(plan, a.view(R, H * D), a8, as_)
    tdp.tdp_matmul8(plan, a8, as_, o8, os, out, res=h)

    import block_ref
    segs, _ = block_ref.segments(B, dims, tiles, overlap)
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    freq, axis, _ = tdp.tdp_rope_freqs((12, 10, 10))
    hd = n(x) + n(res)
    y = ref.rms_norm(hd, n(w), 1e-6)[2]
    qd = ref.turn((y @ n(wq).T).reshape(R, H, D), ref.angles(segs, P.cpu().numpy(), freq, axis, True)[1], 1.0, False)[0]
    csegs = [(0, b, b * S, S) for b in range(B)]
    kd = ref.turn(n(k).reshape(B * S, H, D), ref.angles(csegs, Pc.cpu().numpy().reshape(-1), freq, axis, True)[1], 1.0, False)[0].reshape(B, S, H, D)
    ad = block_ref.xattn(segs, qd, kd, n(v), keep.cpu().numpy(), D ** -0.5)[0]["out"][0]
    part = ad.reshape(R, -1) @ n(wo).T
    err = n(out) - hd - part
    # e4m3 twice through y and wq into scores of spread one, and twice in the last product: four times 0.027 in the mean square
    assert np.linalg.norm(err) < 4 * 0.027 * np.linalg.norm(part) + 2.0 ** -8 * np.linalg.norm(hd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,N", [(9, 264), (70, 520), (500, 1032), (20000, 264)])
def test_scales_of_any_size(tdp, dtype, rows, N):
    """Rows and weights whose scales are no middling numbers, from the smallest float to those of rows of the largest: the product of
    both scales and the sum is as exact as any where it is a float itself, infinite past that.  The bound counts the sum's roundings, four
    behind it and the smallest float's step."""
    import torch
    K, dt = 528, torch.float32 if dtype == "f32" else torch.bfloat16
    x8, xs, w8, ws, b, s = _case(rows, K, N, dt)
    far = torch.tensor([2.0 ** -149, 2.0 ** -130, 2.0 ** -109, 1e-20, 1.0, 1e20, 2.0 ** 90, 1e34, 2.0 ** 119, 3e38, 0.0], device="cuda")
    row, ch = torch.arange(rows, device="cuda"), torch.arange(N, device="cuda")
    xs = torch.where(row % 2 == 1, far[row % 11], xs)
    ws = torch.where(ch % 3 == 1, far[ch % 11], ws)
    # whole small numbers, exact in any order, some of them 0
    z = torch.randint(-2, 3, (N, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows)).float()
    z[::5, 2:] = 0
    w8 = torch.where((ch % 2 == 0)[:, None], z, w8.float()).to(torch.float8_e4m3fn)
    out = torch.empty(rows, N, dtype=dt, device="cuda")
    for bias, res in ((None, None), (b, s)):
        tdp.tdp_matmul8(_plan(tdp, dtype), x8, xs, w8, ws, out, bias=bias, res=res)
        x, w = x8.double() * xs.double()[:, None], w8.double() * ws.double()[:, None]
        want, size = x @ w.T, x.abs() @ w.abs().T
        if res is not None:
            want, size = want + b.double() + s.double(), size + b.double().abs() + s.double().abs()
        tol = 2 * (K + 8) * U * size + 8 * 2.0 ** -149 + (2.0 ** -8 * want.abs() + 2.0 ** -133 if dtype == "bf16" else 0)
        most, got = float(torch.finfo(dt).max), out.double()
        inside, past = want.abs() + tol < most, want.abs() - tol > most * (1 + 2.0 ** -8)
        assert int(inside.sum()) > rows * N // 2 and int(past.sum()) > 0
        assert ((got - want).abs() <= tol)[inside].all()
        assert (got == torch.copysign(torch.full_like(want, float("inf")), want))[past].all()
