"""Group normalisation of groups that hold one value over and over: mean is that value and nothing is left of the rows."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("level", [0.1, -3.3, 1000.1, 123456.7])
@pytest.mark.parametrize("C,G", [(16, 4), (120, 20), (128, 32), (48, 1), (1280, 32), (4096, 1)])
@pytest.mark.parametrize("dims", [(1, 1, 3), (3, 17, 23), (5, 40, 37)])
def test_constant_groups(tdp, dtype, level, C, G, dims):
    """Deviations from the value are zero and so is their sum, however the value's own multiples round.  rstd is a square
    root and a quotient of eps: 2^-22 of it."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    plan = tdp.tdp_plan_create(2, *dims, 8, dtype, (1, 1, 1), (0, 0, 0))
    R = plan.B * plan.total_tile_tokens
    x = torch.full((R, C), level, dtype=dt, device="cuda")
    x[R // 2:] *= -0.7
    y, mean, rstd = torch.empty_like(x), torch.empty(1, 2, G, device="cuda"), torch.empty(1, 2, G, device="cuda")
    tdp.tdp_group_norm(plan, x, G, None, None, y, mean, rstd, eps=1e-5)
    assert torch.equal(mean[0], x.float()[[0, R - 1]][:, :1].expand(2, G))
    assert (y == 0).all()
    assert (rstd.double() * 1e-5 ** 0.5 - 1).abs().max() <= 2.0 ** -22
