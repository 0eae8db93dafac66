"""The operators together: a block's outputs and gradients against plain torch in 64 bits, and the example."""
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


def test_block_against_plain_torch(tdp):
    """fp32, ragged tiles, a mask by tile and dropout: outputs and every gradient.  The plain form is torch's autograd
    in 64 bits over explicit (tile, item) loops.  Each of the chain's seven operators rounds at 2^-24 of its terms, sums of
    up to a thousand of them: 2^-24 * 2^10 of the largest value, with room for the growth through the chain."""
    import torch
    from blend_tdp_tile_gb300.block import TileBlock
    torch.manual_seed(3)
    B, dims, tiles, overlap = 2, (3, 7, 10), (1, 2, 2), (0, 1, 2)
    segs, R = ref.segments(B, dims, tiles, overlap)
    plan = tdp.tdp_plan_create(B, *dims, 8, "f32", tiles, overlap)
    C, S, ctx, p = 24, 37, 20, 0.3
    block = TileBlock(C, heads=4, kv_heads=2, head_dim=16, context=ctx, groups=6, p=p, dtype=torch.float32)
    with torch.no_grad():
        block.gamma.normal_(1, 0.2)
        block.beta.normal_(0, 0.2)
    x = torch.randn(R, C, device="cuda", requires_grad=True)
    states = torch.randn(B, S, ctx, device="cuda", requires_grad=True)
    mask = torch.rand(plan.n_tiles, B, S, device="cuda") < 0.5
    mask[1, 0] = False
    rng = torch.tensor([99, 7], dtype=torch.int64, device="cuda")
    w = torch.randn(R, C, device="cuda")
    y = block(plan, x, states, mask, rng)
    rng[1] += 1                                  # moved on before the gradient, which keeps its own
    (y * w).sum().backward()
    got = {"y": y, "x": x.grad, "states": states.grad} | {n: q.grad for n, q in block.named_parameters()}

    P = {n: q.detach().double().cpu().requires_grad_() for n, q in block.named_parameters()}
    xd, sd = x.detach().double().cpu().requires_grad_(), states.detach().double().cpu().requires_grad_()
    keep = torch.from_numpy((ref.philox(R * C, 99, 7) >= np.uint64(round(p * 2 ** 32))).reshape(R, C))
    rows = []
    for t, b, r0, T in segs:
        xs = xd[r0:r0 + T]
        g = xs.reshape(T, 6, 4)
        h = ((g - g.mean((0, 2), keepdim=True)) / (g.var((0, 2), correction=0, keepdim=True) + 1e-5).sqrt()).reshape(T, C)
        h = torch.nn.functional.silu(h * P["gamma"] + P["beta"])
        q = (h @ P["to_q.weight"].T).reshape(T, 4, 16)
        kv = (sd[b] @ P["to_kv.weight"].T).reshape(S, 2, 2, 16).repeat_interleave(2, 2)
        on = mask[t, b].cpu()
        s = torch.einsum("thd,shd->hts", q, kv[on, 0]) / 4
        a = torch.einsum("hts,shd->thd", s.softmax(-1), kv[on, 1]).reshape(T, 64) if on.any() else xs.new_zeros(T, 64)
        rows.append(xs + torch.where(keep[r0:r0 + T], (a @ P["to_out.weight"].T) / (1 - p), 0))
    yd = torch.cat(rows)
    (yd * w.double().cpu()).sum().backward()
    want = {"y": yd, "x": xd.grad, "states": sd.grad} | {n: q.grad for n, q in P.items()}
    for n, v in want.items():
        err = float((got[n].detach().double().cpu() - v.detach()).abs().max() / v.detach().abs().max())
        assert err < 2.0 ** -24 * 2 ** 10, (n, err)


@pytest.mark.parametrize("name", ["tiny", "small"])
def test_example_runs_and_learns(tdp, name):
    import importlib.util
    import os
    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tile_block.py")
    spec = importlib.util.spec_from_file_location("tile_block_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    Z, losses = mod.run(name, steps=6, log=lambda *_: None)
    assert torch.isfinite(Z.float()).all() and losses[-1] < losses[0]


def test_kept_workspaces(tdp):
    """A plan's small workspace serves calls of one stream; two streams at once and a graph use their own."""
    import torch
    plan = tdp.tdp_plan_create(1, 5, 9, 14, 8, "f32", (2, 2, 2), (2, 3, 3))
    R, C, G = plan.B * plan.total_tile_tokens, 64, 8
    x = [torch.randn(R, C, device="cuda") + i for i in range(2)]
    stat = lambda: torch.empty(plan.n_tiles * plan.B * G, device="cuda")  # noqa: E731
    y, st = [torch.empty_like(t) for t in x], [(stat(), stat()) for _ in x]
    want = []
    for t in x:
        o = torch.empty_like(t)
        tdp.tdp_group_norm(plan, t, G, None, None, o, stat(), stat())
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(50):
        for t, o, s, m in zip(x, y, streams, st):
            with torch.cuda.stream(s):
                tdp.tdp_group_norm(plan, t, G, None, None, o, *m)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(y, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tdp.tdp_group_norm(plan, x[0], G, None, None, y[0], *st[0])
    y[0].fill_(0)
    for _ in range(20):         # replays beside calls of another stream
        with torch.cuda.stream(streams[0]):
            graph.replay()
        tdp.tdp_group_norm(plan, x[1], G, None, None, y[1], *st[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(y, want))
