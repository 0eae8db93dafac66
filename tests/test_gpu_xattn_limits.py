"""Cross attention of half a million tiles of one token: tens of millions of items a launch."""
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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_tiles_and_heads(tdp, dtype):
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    B, H, D, S = 2, 64, 8, 77
    plan = tdp.tdp_plan_create(B, 64, 64, 64, 8, dtype, (64, 64, 64), (0, 0, 0))
    R = B * plan.total_tile_tokens                      # row t * B + b
    g = torch.Generator(device="cuda").manual_seed(0)
    t = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    q, k, v, dout = t(R, H, D), t(B, S, H, D), t(B, S, H, D), t(R, H, D)
    out, lse, dq, dk, dv = torch.empty_like(q), torch.empty(R, H, device="cuda"), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    tdp.tdp_cross_attn(plan, q, k, v, None, out, lse)
    tdp.tdp_cross_attn_grad(plan, q, k, v, None, out, lse, dout, dq, dk, dv)
    h = lambda x: x.double().cpu().numpy()  # noqa: E731
    rows = np.unique(np.concatenate([np.arange(6), R - 1 - np.arange(6), np.random.default_rng(0).integers(0, R, 200)]))
    segs = [(0, int(r) % B, i, 1) for i, r in enumerate(rows)]
    want, smax = ref.xattn(segs, h(q[rows]), h(k), h(v), None, 1 / math.sqrt(D), h(dout[rows]))
    for name, x in (("out", out), ("lse", lse), ("dq", dq)):
        val, mag = want[name]
        u = ref.xattn_unit("f32" if name == "lse" else dtype, D, smax)
        assert (np.abs(h(x[rows]) - val) <= u * mag + 1e-30).all(), name
    # dk and dv are sums over a quarter of a million rows: whole, in 64 bits, head by head.  Terms are rounded to bf16 once,
    # results once (2^-8 / sqrt(3) in the mean square, and their like in dS for dk); fp32 sums of 2^18 terms in order err by
    # 2^-24 * 2^9 of them if their roundings are random, eight times that at most.
    tol = 2 * 2.0 ** -8 / 3 ** 0.5 if dtype == "bf16" else 2.0 ** -12
    for head in (0, 37, H - 1):
        for b in range(B):
            x, go, kk, vv = q[b::B, head].double(), dout[b::B, head].double(), k[b, :, head].double(), v[b, :, head].double()
            p = (x @ kk.T / math.sqrt(D)).softmax(-1)
            dp = go @ vv.T
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(D)
            for name, d, w in (("dk", dk, ds.T @ x), ("dv", dv, p.T @ go)):
                err = float((d[b, :, head].double() - w).norm() / w.norm())
                assert err < tol, (name, head, b, err)
