"""Cross attention of many query heads on a key head, and the whole error of long sums."""
import math

import numpy as np
import pytest

import block_ref as ref
from test_gpu_xattn import FLAT, RAGGED, one, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [127, 128, 130, 131, 256])
@pytest.mark.parametrize("kind", ["none", "holes", "tile"])
def test_groups_of_many_heads(tdp, dtype, G, kind):
    """Groups of more than 128 heads are head blocks of their largest divisor up to 128: two of 65, two of 128, or one by one."""
    run(tdp, (2, (1, 5, 7), (1, 2, 2), (0, 1, 2)), dtype, G, 1, 16, 150, kind, True)
    run(tdp, (1, (2, 4, 5), (1, 1, 1), (0, 0, 0)), dtype, 2 * G, 2, 72, 130, "length" if kind == "tile" else kind, True, seed=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,kind", [(1000, "none"), (1000, "holes"), (5000, "none"), (5000, "left")])
@pytest.mark.parametrize("geom", [one(1, B=2), one(40, B=2), RAGGED, FLAT], ids=["token", "forty", "ragged", "flat"])
@pytest.mark.parametrize("D", [64, 128])
def test_whole_error_of_long_sums(tdp, dtype, S, kind, geom, D):
    """A bound on the norm of the error sees a single state in a thousand lost (3 %), where one by magnitudes does not.
    bf16: a probability and the output are rounded once, each by 2^-8 / sqrt(3) in the mean square at most, independently.
    fp32: sums of S products of D roundings: 2^-24 * sqrt(S) if they are random, and the scores' own D * 2^-24 in the
    exponent; four times that."""
    import torch
    B, dims, tiles, overlap = geom
    segs, R = ref.segments(*geom)
    rng = np.random.default_rng(S + D)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    t = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).to(dt).cuda()  # noqa: E731
    q, k, v = t(R, 4, D), t(B, S, 2, D), t(B, S, 2, D)
    mask = None
    if kind == "holes":
        mask = rng.random((B, S)) < 0.7
    elif kind == "left":
        mask = np.arange(S) >= np.array([S // 3, S - 900])[:B, None]
    want, _ = ref.xattn(segs, *(x.double().cpu().numpy() for x in (q, k, v)), mask, 1 / math.sqrt(D))
    plan = tdp.tdp_plan_create(B, *dims, 8, dtype, tiles, overlap)
    out = torch.empty_like(q)
    tdp.tdp_cross_attn(plan, q, k, v, None if mask is None else torch.from_numpy(mask).cuda(), out)
    val = want["out"][0]
    err = np.linalg.norm(out.double().cpu().numpy() - val) / np.linalg.norm(val)
    assert err < (math.sqrt(2) * 2.0 ** -8 / math.sqrt(3) if dtype == "bf16" else 4 * 2.0 ** -24 * (math.sqrt(S) + D))
