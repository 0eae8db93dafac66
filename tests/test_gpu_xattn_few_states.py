"""bf16 gradients of rows that keep few states: as exact wherever the states lie."""
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


def _places(kind, n, S):
    """n kept states: together across a 128-state boundary, at both ends (a run that wraps), or spread out."""
    if kind == "across":
        return np.arange(128 - n // 2, 128 - n // 2 + n)
    if kind == "wrapped":
        return (np.arange(n) - n // 2) % S
    return np.linspace(0, S - 1, n).round().astype(int)


@pytest.mark.parametrize("n", [2, 4, 9, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["across", "wrapped", "spread"])
@pytest.mark.parametrize("per_tile", [False, True])
def test_few_states_in_several_tiles(tdp, n, D, kind, per_tile):
    """dP and delta nearly cancel.  dS and the gradient are each rounded to bf16 once: a rounding's error is uniform over
    half a spacing, at most 2^-8 / sqrt(3) in the mean square, and two of them are independent."""
    import torch
    B, dims, tiles, overlap = 2, (3, 8, 12), (1, 2, 2), (0, 2, 2)
    segs, R = ref.segments(B, dims, tiles, overlap)
    nt, S, H, K = len(segs) // B, 700, 8, 4
    rng = np.random.default_rng(n)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).bfloat16().cuda()  # noqa: E731
    q, k, v, dout = t(R, H, D), t(B, S, K, D), t(B, S, K, D), t(R, H, D)
    mask = np.zeros((nt, B, S) if per_tile else (B, S), bool)
    mask[..., _places(kind, n, S)] = True
    if per_tile:
        mask[1:] = False
        mask[1:, :, 200:600] = True             # other tiles keep many, and the first none of them
    want, _ = ref.xattn(segs, *(x.double().cpu().numpy() for x in (q, k, v)), mask, 1 / math.sqrt(D), dout.double().cpu().numpy())
    md = torch.from_numpy(mask).cuda()
    gone = ~md.reshape(-1, B, S).any(0)
    k[gone], v[gone] = float("nan"), float("inf")
    plan = tdp.tdp_plan_create(B, *dims, 8, "bf16", tiles, overlap)
    got = []
    for _ in range(2):
        out, lse, dq, dk, dv = torch.empty_like(q), torch.empty((R, H), device="cuda"), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        tdp.tdp_cross_attn(plan, q, k, v, md, out, lse)
        tdp.tdp_cross_attn_grad(plan, q, k, v, md, out, lse, dout, dq, dk, dv)
        got.append((dq, dk, dv))
    few = np.zeros(R, bool)
    for tile, b, r0, T in segs:
        few[r0:r0 + T] = not per_tile or tile == 0
    parts = {"dq": (few,), "dq of others": (~few,), "dk": (slice(None),), "dv": (slice(None),)}
    for name, at in parts.items():
        i = {"dq": 0, "dk": 1, "dv": 2}[name[:2]]
        assert torch.equal(got[0][i], got[1][i])
        val = want[name[:2]][0][at]
        if not val.size:
            continue
        err = np.linalg.norm(got[0][i].double().cpu().numpy()[at] - val) / np.linalg.norm(val)
        assert err < math.sqrt(2) * 2.0**-8 / math.sqrt(3), (name, err)
