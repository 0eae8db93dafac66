"""Refusals of the per-tile block's operators: every invalid argument is turned into a status or an
exception on the host, before any launch."""
import ctypes
import os

import numpy as np
import pytest

from test_abi_host import no_gpu_only, tdp  # noqa: F401  (fixture)

P = 4096          # an aligned address that is never read


def _shape(tdp, **kw):
    a = tdp._XAttn()
    base = dict(q_heads=4, kv_heads=2, head_dim=64, states=10, mask_per_tile=0, scale=0.125, q_row=256, q_head=64,
                k_item=1280, k_state=128, k_head=64, v_item=1280, v_state=128, v_head=64)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def _plan(tdp, dtype="bf16", B=1):
    return tdp.tdp_plan_create(B, 3, 8, 12, 16, dtype, (1, 2, 2), (0, 2, 2))


def _lib(tdp):
    return tdp._lib


@pytest.mark.parametrize("kw,status", [
    (dict(q_heads=0), 1), (dict(kv_heads=0), 1), (dict(q_heads=3), 1), (dict(head_dim=0), 1), (dict(states=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(k_state=-128), 1),
    (dict(head_dim=136), 5), (dict(states=(1 << 20) + 1), 5),
    (dict(head_dim=60), 4), (dict(q_row=252), 4), (dict(v_head=1), 4), (dict(k_item=2), 4),
    (dict(q_heads=1 << 24, kv_heads=1 << 23), 5), (dict(k_item=1 << 38), 5),
    (dict(q_row=0), 1), (dict(q_head=0), 1), (dict(k_state=0), 1), (dict(v_state=0), 1),
])
def test_cross_attn_shapes_refused(tdp, kw, status):  # noqa: F811
    n = ctypes.c_int64()
    a = _shape(tdp, **kw)
    assert _lib(tdp).tdp_cross_attn_workspace(_plan(tdp).handle, ctypes.byref(a), 0, ctypes.byref(n)) == status
    assert tdp.tdp_last_error_detail()


@no_gpu_only
def test_cross_attn_buffers_refused(tdp):  # noqa: F811
    lib, plan, a = _lib(tdp), _plan(tdp), _shape(tdp)
    n = ctypes.c_int64()
    assert lib.tdp_cross_attn_workspace(plan.handle, ctypes.byref(a), 1, ctypes.byref(n)) == 0 and n.value > 0

    def fwd(h=plan.handle, shape=ctypes.byref(a), **kw):
        b = dict(q=P, k=P, v=P, mask=None, out=P, lse=None, ws=P, n=1 << 30) | kw
        return lib.tdp_cross_attn(h, shape, b["q"], b["k"], b["v"], b["mask"], b["out"], b["lse"], b["ws"], b["n"], None)

    def grad(**kw):
        b = dict(q=P, k=P, v=P, mask=None, out=P, lse=P, dout=P, dq=P, dk=P, dv=P, ws=P, n=n.value) | kw
        return lib.tdp_cross_attn_grad(plan.handle, ctypes.byref(a), b["q"], b["k"], b["v"], b["mask"], b["out"], b["lse"],
                                       b["dout"], b["dq"], b["dk"], b["dv"], b["ws"], b["n"], None)
    assert fwd(h=None) == 1 and fwd(shape=None) == 1
    assert [fwd(**{x: None}) for x in ("q", "k", "v", "out")] == [1] * 4
    assert [fwd(**{x: P + 8}) for x in ("q", "k", "v", "out")] == [4] * 4
    assert fwd(lse=P + 2) == 4 and fwd(ws=P + 16) == 4
    assert [grad(**{x: None}) for x in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws")] == [1] * 10
    assert [grad(**{x: P + 8}) for x in ("q", "k", "v", "out", "dout", "dq", "dk", "dv", "ws")] == [4] * 9
    assert grad(n=n.value - 1) == 1
    # a split over the states needs its workspace
    one = tdp.tdp_plan_create(1, 1, 1, 1, 16, "bf16", (1, 1, 1), (0, 0, 0))
    b = _shape(tdp, states=4096, k_item=4096 * 128, v_item=4096 * 128)
    assert lib.tdp_cross_attn_workspace(one.handle, ctypes.byref(b), 0, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.tdp_cross_attn(one.handle, ctypes.byref(b), P, P, P, None, P, None, None, 0, None) == 1
    # no items: nothing to do, nothing read
    none = _plan(tdp, B=0)
    assert lib.tdp_cross_attn(none.handle, ctypes.byref(a), None, None, None, None, None, None, None, 0, None) == 0
    assert lib.tdp_cross_attn_grad(none.handle, ctypes.byref(a), *[None] * 11, 0, None) == 0


@pytest.mark.parametrize("C,groups,status", [(0, 1, 1), (16, 0, 1), (16, 3, 1), (4, 1, 4), (12, 3, 4), (-8, 1, 1)])
def test_group_norm_shapes_refused(tdp, C, groups, status):  # noqa: F811
    n = ctypes.c_int64()
    assert _lib(tdp).tdp_group_norm_workspace(_plan(tdp).handle, C, groups, ctypes.byref(n)) == status


@no_gpu_only
def test_group_norm_buffers_refused(tdp):  # noqa: F811
    lib, plan = _lib(tdp), _plan(tdp)
    need = tdp.tdp_group_norm_workspace(plan, 16, 4)

    def fwd(eps=1e-5, act=1, **kw):
        b = dict(x=P, gamma=P, beta=P, y=P, mean=P, rstd=P, ws=P, n=need) | kw
        return lib.tdp_group_norm(plan.handle, 16, 4, eps, act, b["x"], b["gamma"], b["beta"], b["y"], b["mean"], b["rstd"],
                                  b["ws"], b["n"], None)

    def grad(act=1, **kw):
        b = dict(x=P, gamma=P, beta=P, mean=P, rstd=P, dy=P, dx=P, dgamma=P, dbeta=P, ws=P, n=need) | kw
        return lib.tdp_group_norm_grad(plan.handle, 16, 4, act, b["x"], b["gamma"], b["beta"], b["mean"], b["rstd"], b["dy"],
                                       b["dx"], b["dgamma"], b["dbeta"], b["ws"], b["n"], None)
    assert fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1 and fwd(act=2) == 1 and grad(act=-1) == 1
    assert [fwd(**{k: None}) for k in ("x", "y", "mean", "rstd", "ws")] == [1] * 5
    assert [fwd(**{k: P + 8}) for k in ("x", "gamma", "beta", "y", "ws")] == [4] * 5
    assert fwd(mean=P + 2) == 4 and fwd(n=need - 1) == 1
    assert [grad(**{k: None}) for k in ("x", "mean", "rstd", "dy", "dx", "ws", "dgamma", "dbeta")] == [1] * 8
    assert [grad(**{k: P + 2}) for k in ("x", "gamma", "beta", "mean", "rstd", "dy", "dx", "dgamma", "dbeta", "ws")] == [4] * 10
    assert grad(n=need - 1) == 1
    assert lib.tdp_group_norm(_plan(tdp, B=0).handle, 16, 4, 0.1, 0, *[None] * 7, 0, None) == 0
    assert lib.tdp_group_norm(None, 16, 4, 0.1, 0, *[None] * 7, 0, None) == 1


@no_gpu_only
def test_dropout_refused(tdp):  # noqa: F811
    lib, plan = _lib(tdp), _plan(tdp)
    add = lambda n=8, p=0.1, rng=P, x=P, res=None, out=P, h=plan.handle: lib.tdp_dropout_add(h, n, p, rng, x, res, out, None)  # noqa: E731
    assert add(h=None) == 1 and add(n=-1) == 1 and add(p=-0.1) == 1 and add(p=1.5) == 1 and add(p=float("nan")) == 1
    assert add(rng=None) == 1 and add(x=None) == 1 and add(out=None) == 1
    assert add(rng=P + 4) == 4 and add(x=P + 8) == 4 and add(res=P + 2) == 4 and add(out=P + 8) == 4
    assert add(n=1 << 60) == 5
    assert add(n=0, rng=None, x=None, out=None) == 0
    assert lib.tdp_dropout_grad(plan.handle, 8, 2.0, P, P, P, None) == 1
    assert lib.tdp_dropout_grad(plan.handle, 8, 0.5, P, None, P, None) == 1


def test_binding_refuses_on_the_host(tdp):  # noqa: F811
    torch = pytest.importorskip("torch")
    plan = _plan(tdp, "f32")
    R = plan.total_tile_tokens
    q, k = torch.zeros(R, 2, 64), torch.zeros(1, 5, 2, 64)
    with pytest.raises(ValueError):
        tdp.tdp_cross_attn(plan, q, k, k, None, q)                  # CPU tensors
    with pytest.raises(ValueError):
        tdp.tdp_cross_attn(plan, q[0], k, k, None, q)
    with pytest.raises(TypeError):
        tdp._strides(np.zeros(3), "q", (3,), ())
    with pytest.raises(ValueError):
        tdp.tdp_group_norm(plan, torch.zeros(R, 16), 4, None, None, torch.zeros(R, 16), None, None)
    with pytest.raises(ValueError):
        tdp._act("gelu")
    with pytest.raises(ValueError):
        tdp.tdp_dropout_add(plan, torch.zeros(8), None, 0.5, torch.zeros(2, dtype=torch.int64), torch.zeros(8))


def test_header_and_binding_agree(tdp):  # noqa: F811
    src = open(os.path.join(os.path.dirname(tdp.LIB_PATH), "..", "include", "tdp.h")).read()
    assert f"#define TDP_MAX_HEAD_DIM {tdp.TDP_MAX_HEAD_DIM}" in src and "#define TDP_MAX_STATES (1 << 20)" in src
    assert tdp.TDP_MAX_STATES == 1 << 20 and ctypes.sizeof(tdp._XAttn) == 24 + 8 * 8
