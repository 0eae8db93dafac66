"""Sizes that cross attention takes up to its stated limit, R * q_heads below 2^31; on the host, without a launch."""
import ctypes

import pytest

from test_abi_host import tdp  # noqa: F401  (fixture)


def _status(tdp, plan, Hq, Hkv, D, S, per_tile, grad):  # noqa: F811
    a, n = tdp._XAttn(), ctypes.c_int64()
    v = dict(q_heads=Hq, kv_heads=Hkv, head_dim=D, states=S, mask_per_tile=per_tile, scale=1.0, q_row=Hq * D, q_head=D,
             k_item=S * Hkv * D, k_state=Hkv * D, k_head=D, v_item=S * Hkv * D, v_state=Hkv * D, v_head=D)
    for k, x in v.items():
        setattr(a, k, x)
    return tdp._lib.tdp_cross_attn_workspace(plan.handle, ctypes.byref(a), grad, ctypes.byref(n)), n.value


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("B,dims,Hq,Hkv,per_tile", [
    (2, (64, 64, 64), 64, 64, 0), (1, (64, 64, 64), 128, 128, 1), (16, (64, 64, 64), 128, 32, 1), (3, (65, 65, 65), 160, 40, 0),
    (1, (128, 1024, 1024), 8, 8, 0), (1, (128, 1024, 1024), 15, 3, 1)])
def test_every_size_below_the_limit(tdp, dtype, grad, B, dims, Hq, Hkv, per_tile):  # noqa: F811
    plan = tdp.tdp_plan_create(B, *dims, 8, dtype, (64, 64, 64) if max(dims) < 128 else (2, 2, 2), (0, 0, 0))
    assert B * plan.total_tile_tokens * Hq < 1 << 31
    assert _status(tdp, plan, Hq, Hkv, 64, 77, per_tile, grad)[0] == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_past_the_limit(tdp, dtype):  # noqa: F811
    plan = tdp.tdp_plan_create(1, 128, 1024, 1024, 8, dtype, (2, 2, 2), (0, 0, 0))
    assert _status(tdp, plan, 16, 16, 64, 77, 0, 0)[0] == 5
    assert _status(tdp, plan, 1 << 20, 1, 8, 77, 0, 1)[0] == 5
