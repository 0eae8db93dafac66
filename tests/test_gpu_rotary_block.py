"""The block of the norm, rotary positions and attention to conditioning tokens: outputs and gradients against plain torch in 64
bits, its 8-bit form, and the example."""
import numpy as np
import pytest

import block_ref
import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


B, DIMS, TILES, OVERLAP = 2, (3, 7, 10), (1, 2, 2), (0, 1, 2)
C, S, CTX, H, K, D, PAIRS = 32, 37, 48, 4, 2, 16, (3, 2, 1)


def _make(tdp, dtype, **kw):
    import torch
    from blend_tdp_tile_gb300.block import RotaryBlock
    torch.manual_seed(3)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    segs, R = block_ref.segments(B, DIMS, TILES, OVERLAP)
    plan, tokens_plan = tdp.tdp_plan_create(B, *DIMS, 8, dtype, TILES, OVERLAP), tdp.tdp_plan_create(B, 1, 1, S, 8, dtype, (1, 1, 1), (0, 0, 0))
    block = RotaryBlock(C, H, K, D, CTX, PAIRS, dtype=dt, **kw)
    with torch.no_grad():
        block.w.normal_(1, 0.2)
    x = torch.randn(R, C, device="cuda").to(dt).requires_grad_()
    tokens = torch.randn(B, S, CTX, device="cuda").to(dt).requires_grad_()
    Q = torch.randint(0, 40, (6 * R,), dtype=torch.int32, device="cuda")
    P = torch.randint(-8, 40, (B, 3, S, 2), dtype=torch.int32, device="cuda")
    mask = torch.rand(plan.n_tiles, B, S, device="cuda") < 0.5
    mask[1, 0] = False
    return plan, tokens_plan, segs, R, block, x, tokens, Q, P, mask


def _plain(tdp, segs, R, block, x, tokens, Q, P, mask, keep=None, p=0.0):
    """The block in 64 bits over explicit (tile, item) loops."""
    import torch
    W = {n: q.detach().double().cpu().requires_grad_() for n, q in block.named_parameters()}
    xd, td = x.detach().double().cpu().requires_grad_(), tokens.detach().double().cpu().requires_grad_()
    freq, axis, _ = tdp.tdp_rope_freqs(PAIRS)
    aq = torch.from_numpy(ref.angles(segs, Q.cpu().numpy(), freq, axis, True)[1])
    ak = torch.from_numpy(ref.angles([(0, b, b * S, S) for b in range(B)], P.cpu().numpy().reshape(-1), freq, axis, True)[1])

    def turn(v, angle):
        n = angle.shape[1]
        a, b, c, s = v[..., :n], v[..., n:2 * n], angle.cos()[:, None], angle.sin()[:, None]
        return torch.cat((a * c - b * s, a * s + b * c, v[..., 2 * n:]), -1)
    y = xd * (xd.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * W["w"]
    q = turn((y @ W["to_q.weight"].T).reshape(R, H, D), aq)
    kv = (td @ W["to_kv.weight"].T).reshape(B * S, 2, K, D)
    k, v = turn(kv[:, 0], ak).reshape(B, S, K, D).repeat_interleave(H // K, 2), kv[:, 1].reshape(B, S, K, D).repeat_interleave(H // K, 2)
    rows = []
    for t, b, r0, T in segs:
        on = mask[t, b].cpu()
        if on.any():
            a = torch.einsum("hts,shd->thd", (torch.einsum("thd,shd->hts", q[r0:r0 + T], k[b, on]) / D ** 0.5).softmax(-1), v[b, on]).reshape(T, H * D)
        else:
            a = q.new_zeros(T, H * D)
        rows.append(a @ W["to_out.weight"].T)
    a = torch.cat(rows)
    out = xd + (torch.where(keep, a / (1 - p), 0) if keep is not None else a)
    return out, xd, td, W


def test_block_against_plain_torch(tdp):
    """fp32, ragged tiles, a mask by tile and dropout.  Each of the chain's nine operators rounds at 2^-24 of its terms, sums of up to
    a thousand of them: 2^-24 * 2^10 of the largest value, with room for the growth through the chain."""
    import torch
    p = 0.3
    plan, tokens_plan, segs, R, block, x, tokens, Q, P, mask = _make(tdp, "f32", p=p)
    rng = torch.tensor([99, 7], dtype=torch.int64, device="cuda")
    w = torch.randn(R, C, device="cuda")
    y = block(plan, x, Q, tokens_plan, tokens, P, mask, rng)
    rng[1] += 1
    (y * w).sum().backward()
    got = {"y": y, "x": x.grad, "tokens": tokens.grad} | {n: q.grad for n, q in block.named_parameters()}
    keep = torch.from_numpy((block_ref.philox(R * C, 99, 7) >= np.uint64(round(p * 2 ** 32))).reshape(R, C))
    yd, xd, td, W = _plain(tdp, segs, R, block, x, tokens, Q, P, mask, keep, p)
    (yd * w.double().cpu()).sum().backward()
    want = {"y": yd, "x": xd.grad, "tokens": td.grad} | {n: q.grad for n, q in W.items()}
    for n, v in want.items():
        err = float((got[n].detach().double().cpu() - v.detach()).abs().max() / v.detach().abs().max())
        assert err < 2.0 ** -24 * 2 ** 10, (n, err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_checkpoints_in_8_bits(tdp, dtype):
    """The same outputs, to the bit; gradients of the norm from e4m3's rows, whose values are up to 2^-4 off and 0.027 in the mean
    square: w's is that much off, x's less (only the mean's part reads them), and nothing behind the norm changes."""
    import torch
    plan, tokens_plan, segs, R, block, x, tokens, Q, P, mask = _make(tdp, dtype)
    w = torch.randn(R, C, device="cuda").to(x.dtype)
    grads = []
    for keep8 in (False, True):
        block.keep8 = keep8
        y = block(plan, x, Q, tokens_plan, tokens, P, mask)
        (y * w).sum().backward()
        grads.append({"y": y.detach().clone(), "x": x.grad, "tokens": tokens.grad} | {n: q.grad for n, q in block.named_parameters()})
        x.grad = tokens.grad = None
        for q in block.parameters():
            q.grad = None
    for n, v in grads[0].items():
        if n in ("x", "w"):
            assert float((grads[1][n].float() - v.float()).norm()) < 0.06 * float(v.float().norm()), n
        else:
            assert torch.equal(grads[1][n], v), n


def test_gradients_captured_while_an_eager_graph_lives(tdp):
    """Forward and gradient of the norm and the rotation as a CUDA graph, of tensors that are leaves of their own: replays give
    the eager call's gradients, and an eager graph of other leaves lives beside it."""
    import torch
    from blend_tdp_tile_gb300.block import rms_norm, rope
    plan, _, _, R, _, x, _, Q, _, _ = _make(tdp, "f32")
    table = tdp.tdp_rope_table(*tdp.tdp_rope_freqs((8, 4, 4))[:2]).cuda()
    w = torch.randn(C, device="cuda")
    g = torch.randn(R, 1, C, device="cuda")

    def step(v):
        v, u = v.detach().requires_grad_(), w.detach().requires_grad_()
        y = rope(plan, rms_norm(plan, v, u, keep8=True).view(R, 1, C), Q, table)
        return torch.autograd.grad((y * g).sum(), [v, u])
    alive = rms_norm(plan, x, w)                # an eager graph that has not been run backward yet
    want = step(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    alive.sum().backward()
    assert torch.isfinite(x.grad).all()


def test_block_served_in_8_bits(tdp):
    """Against the full block: queries through two operands of e4m3 (0.027 each in the mean square), tokens' keys and values the same,
    attention's outputs and the last weights again: no more than six such errors of the block's share."""
    import torch
    plan, tokens_plan, segs, R, block, x, tokens, Q, P, mask = _make(tdp, "bf16")
    with torch.no_grad():
        full = block.eval()(plan, x, Q, tokens_plan, tokens, P, mask)
        few = block.to_8bit(plan)(plan, x, Q, tokens_plan, tokens, P, mask)
        share = float((full.float() - x.float()).norm())
        assert 0 < float((few.float() - full.float()).norm()) < 6 * 0.027 * share + 2.0 ** -8 * float(full.float().norm())
    with pytest.raises(RuntimeError, match="no gradient"):
        block(plan, x, Q, tokens_plan, tokens, P, mask)
    block.train()
    assert torch.isfinite(torch.autograd.grad(block(plan, x, Q, tokens_plan, tokens, P, mask).float().sum(), x)[0].float()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_in_8_bits(tdp, dtype):
    """A linear layer with a bias on [items, tokens, channels], and onto a residual: rows and weights rounded to e4m3, 0.027 of the
    product each in the mean square; the same rows given in 8 bits are the same to the bit."""
    import torch
    from blend_tdp_tile_gb300.block import Linear8, quant8
    torch.manual_seed(4)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    plan = tdp.tdp_plan_create(1, 1, 1, 1, 8, dtype, (1, 1, 1), (0, 0, 0))
    full = torch.nn.Linear(144, 200, device="cuda", dtype=dt)
    few = Linear8(plan, full)
    x, res = torch.randn(3, 37, 144, device="cuda").to(dt), torch.randn(3, 37, 200, device="cuda").to(dt)
    with torch.no_grad():
        y, z = few(plan, x), few(plan, x, res=res)
        want = full.double()(x.double())
        product = want - full.bias
        assert y.shape == (3, 37, 200) and y.dtype == dt
        for got, to in ((y, want), (z, want + res.double())):
            assert float((got.double() - to).norm()) < 2 * 0.027 * float(product.norm()) + 2.0 ** -8 * float(to.norm())
        x8, scale = quant8(plan, x)
        assert torch.equal(few(plan, x8, scale), y)
        assert few.w8.dtype == torch.uint8 and torch.equal(few.to("cuda")(plan, x), y)
    with pytest.raises(RuntimeError, match="no gradient"):
        few(plan, x, res=res.requires_grad_())


@pytest.mark.parametrize("name", ["tiny", "small"])
def test_example_runs(tdp, name):
    import importlib.util
    import os
    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "rotary_block.py")
    spec = importlib.util.spec_from_file_location("rotary_block_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    Z8, Z, grads = mod.run(name, steps=2, log=lambda *_: None)
    assert torch.isfinite(Z.float()).all() and torch.isfinite(Z8.float()).all() and not torch.equal(Z, Z8)
    assert set(grads) == {"w", "to_q.weight", "to_kv.weight", "to_out.weight"}
    assert all(torch.isfinite(g.float()).all() and float(g.float().abs().max()) > 0 for g in grads.values())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_changes_of_dtype_leave_8_bits_alone(tdp, dtype):
    """Weights, scales and bias in 8 bits are the same to the bit behind any change of dtype; a block served in 8 bits comes back
    with its weights."""
    import torch
    from blend_tdp_tile_gb300.block import Linear8
    torch.manual_seed(5)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    plan = tdp.tdp_plan_create(1, 1, 1, 1, 8, dtype, (1, 1, 1), (0, 0, 0))
    few, x = Linear8(plan, torch.nn.Linear(144, 200, device="cuda", dtype=dt)), torch.randn(37, 144, device="cuda").to(dt)
    with torch.no_grad():
        want = few(plan, x)
        for change in (lambda: few.to(torch.bfloat16), lambda: few.float(), lambda: few.half().double()):
            change()
            assert torch.equal(few(plan, x), want)
    plan, tokens_plan, segs, R, block, x, tokens, Q, P, mask = _make(tdp, "bf16")
    with torch.no_grad():
        want = block.to_8bit(plan)(plan, x, Q, tokens_plan, tokens, P, mask)
        block.float().bfloat16()
        assert torch.equal(block(plan, x, Q, tokens_plan, tokens, P, mask), want)
