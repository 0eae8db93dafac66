"""Refusals of the norm, the 8-bit products and the rotary positions on the host, and their host-side tables."""
import ctypes
import math
import os
from fractions import Fraction

import numpy as np
import pytest

import linear_ref as ref
from test_abi_host import no_gpu_only, tdp  # noqa: F401  (fixture)

P = 4096          # an aligned address that is never read


def _plan(tdp, dtype="bf16", B=1):
    return tdp.tdp_plan_create(B, 3, 8, 12, 16, dtype, (1, 2, 2), (0, 2, 2))


@no_gpu_only
def test_rms_norm_refused(tdp):  # noqa: F811
    lib, plan = tdp._lib, _plan(tdp)

    def fwd(h=plan.handle, rows=4, C=64, eps=1e-5, **kw):
        b = dict(x=P, res=None, w=P, h=P, y=3 * P, rstd=P, y8=P, ys=P, x8=P, xs=P) | kw
        return lib.tdp_rms_norm(h, rows, C, eps, *b.values(), None)

    def quant(h=plan.handle, rows=4, C=64, x=P, x8=P, xs=P):
        return lib.tdp_quant8(h, rows, C, x, x8, xs, None)
    for f in (fwd, quant):
        assert f(h=None) == 1 and f(rows=-1) == 1 and f(C=0) == 1 and f(C=-8) == 1 and f(x=None) == 1
        assert f(C=60) == 4 and f(C=16392) == 5 and f(C=1 << 30) == 5 and f(rows=1 << 50) == 5
        assert f(x=P + 8) == 4 and f(x8=P + 4) == 4 and f(xs=P + 2) == 4
        assert f(xs=None) == 1 and f(rows=0, x=None, x8=None, xs=None) == 0
    assert fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1 and fwd(eps=float("inf")) == 1
    assert fwd(ys=None) == 1 and fwd(y8=None) == 1 and fwd(x8=None) == 1
    assert fwd(h=plan.handle, y=None, rstd=None, y8=None, ys=None, x8=None, xs=None, **{"res": None}) in (0, 6)     # h alone is an output
    assert lib.tdp_rms_norm(plan.handle, 4, 64, 0.1, P, None, P, *[None] * 7, None) == 1
    assert [fwd(**{k: P + 8}) for k in ("res", "w", "y", "y8")] == [4] * 4 and fwd(rstd=P + 1) == 4 and fwd(ys=P + 2) == 4
    assert quant(x8=None) == 1
    assert lib.tdp_rms_norm(plan.handle, 4, 64, 0.1, P, None, P, 2 * P, 2 * P, *[None] * 5, None) == 1      # h and y in one place


@no_gpu_only
def test_rms_norm_grad_refused(tdp):  # noqa: F811
    lib, plan = tdp._lib, _plan(tdp)
    need = tdp.tdp_rms_norm_grad_workspace(plan, 4, 64)

    def grad(h=plan.handle, rows=4, C=64, **kw):
        b = dict(s=P, x8=None, xs=None, rstd=P, w=P, dy=P, dh=P, dx=P, dw=P, ws=P, n=need) | kw
        return lib.tdp_rms_norm_grad(h, rows, C, *b.values(), None)
    assert need > 0 and grad(h=None) == 1 and grad(rows=-1) == 1 and grad(C=12) == 4 and grad(C=32768) == 5
    assert [grad(**{k: None}) for k in ("s", "rstd", "dy", "dx", "ws")] == [1] * 5
    assert grad(x8=P) == 1 and grad(x8=P, xs=P) == 1 and grad(s=None, x8=P) == 1 and grad(n=need - 1) == 1
    assert [grad(**{k: P + 8}) for k in ("s", "w", "dy", "dh", "dx", "ws")] == [4] * 6 and grad(rstd=P + 2) == 4 and grad(dw=P + 2) == 4
    assert lib.tdp_rms_norm_grad(plan.handle, 0, 64, *[None] * 9, None, 0, None) == 0
    n = ctypes.c_int64()
    assert lib.tdp_rms_norm_grad_workspace(plan.handle, 4, 64, None) == 1 and lib.tdp_rms_norm_grad_workspace(plan.handle, 4, 63, ctypes.byref(n)) == 4


@no_gpu_only
def test_matmul8_refused(tdp):  # noqa: F811
    lib, plan = tdp._lib, _plan(tdp)

    def mm(h=plan.handle, rows=4, K=64, N=64, **kw):
        b = dict(x8=P, xs=P, w8=P, ws=P, bias=P, res=P, out=P) | kw
        return lib.tdp_matmul8(h, rows, K, N, *b.values(), None)
    assert mm(h=None) == 1 and mm(rows=-1) == 1 and mm(K=0) == 1 and mm(N=0) == 1 and mm(N=-8) == 1
    assert mm(K=24) == 4 and mm(N=20) == 4 and mm(K=(1 << 20) + 16) == 5 and mm(N=(1 << 20) + 8) == 5 and mm(rows=(1 << 30) + 1) == 5
    assert mm(rows=1 << 30, N=1 << 20) == 5
    assert [mm(**{k: None}) for k in ("x8", "xs", "w8", "ws", "out")] == [1] * 5
    assert [mm(**{k: P + 8}) for k in ("x8", "w8", "ws", "bias", "res", "out")] == [4] * 6 and mm(xs=P + 2) == 4
    assert lib.tdp_matmul8(plan.handle, 0, 64, 64, *[None] * 7, None) == 0


def _shape(tdp, **kw):
    a = tdp._Rope()
    for k, v in {**dict(heads=4, head_dim=64, rot=32, layout=0, at=1, scale=1.0, x_row=256, x_head=64, out_row=256, out_head=64), **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), 1), (dict(head_dim=0), 1), (dict(rot=0), 1), (dict(rot=31), 1), (dict(rot=66), 1), (dict(layout=2), 1), (dict(at=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(x_row=-8), 1), (dict(out_row=64), 1), (dict(out_head=0), 1), (dict(out_head=32), 1),
    (dict(out_row=200), 1), (dict(out_row=0), 1), (dict(out_row=64, out_head=640), 1), (dict(x_row=512), 1), (dict(x_head=0), 1),
    (dict(heads=1 << 20, out_head=(1 << 38) - 8, x_head=(1 << 38) - 8), 5), (dict(heads=(1 << 20) + 1), 5),
    (dict(head_dim=60, rot=32), 4), (dict(x_row=252), 4), (dict(out_head=65), 4), (dict(head_dim=264), 5), (dict(x_head=1 << 38), 5),
])
@no_gpu_only
def test_rope_shapes_refused(tdp, kw, status):  # noqa: F811
    a = _shape(tdp, **kw)
    for f in (tdp._lib.tdp_rope, tdp._lib.tdp_rope_grad):
        assert f(_plan(tdp).handle, ctypes.byref(a), P, P, P, P, None) == status and tdp.tdp_last_error_detail()


@no_gpu_only
def test_rope_buffers_refused(tdp):  # noqa: F811
    plan, a = _plan(tdp), _shape(tdp)
    for f in (tdp._lib.tdp_rope, tdp._lib.tdp_rope_grad):
        call = lambda h=plan.handle, s=ctypes.byref(a), x=P, q=P, t=P, o=P: f(h, s, x, q, t, o, None)  # noqa: E731
        assert call(h=None) == 1 and call(s=None) == 1 and call(x=None) == 1 and call(q=None) == 1 and call(t=None) == 1 and call(o=None) == 1
        assert call(x=P + 8) == 4 and call(o=P + 8) == 4 and call(q=P + 4) == 4 and call(t=P + 4) == 4
        assert f(_plan(tdp, B=0).handle, ctypes.byref(a), None, None, None, None, None) == 0


PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)


@pytest.mark.parametrize("freq", [1.0, 0.5, 1e-4, 3.3e-9, 1.0 / 3, 12.566370614359172, 1000.25, 2.0 ** 20, -0.7, -1e-5, 0.0, 6.25e-320])
def test_table(tdp, freq):  # noqa: F811
    """freq / 4 pi modulo 1 in whole numbers: two of the last bits hold the axis, and the product is good to 106 bits, of
    which 2^20 / 4 pi takes 17."""
    for axis in range(3):
        got = int(tdp.tdp_rope_table([freq], [axis])[0]) % 2 ** 64
        assert got & 3 == axis
        want = Fraction(freq) / (4 * PI) * 2 ** 64
        off = abs(Fraction(got & ~3) - want % 2 ** 64)
        assert min(off, 2 ** 64 - off) <= 3 + abs(want) / 2 ** 100


def test_table_and_freqs_refused(tdp):  # noqa: F811
    for freq, axis in (([1.0], [3]), ([1.0], [-1]), ([float("nan")], [0]), ([float("inf")], [0]), ([2.0 ** 21], [0])):
        with pytest.raises(tdp.TdpError):
            tdp.tdp_rope_table(freq, axis)
    with pytest.raises(ValueError):
        tdp.tdp_rope_table([1.0, 2.0], [0])
    for kw in (dict(pairs=(-1, 2, 2)), dict(base=0.0), dict(base=float("inf")), dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=float("nan")),
               dict(scaling="yarn", factor=2.0, length=0.0)):
        with pytest.raises(tdp.TdpError):
            tdp.tdp_rope_freqs(**{"pairs": (4, 2, 2), **kw})
    for pairs in ((129, 0, 0), (64, 64, 1), ((1 << 31) - 1,) * 3):
        with pytest.raises(tdp.TdpError) as e:
            tdp.tdp_rope_freqs(pairs)
        assert e.value.status == 5
    with pytest.raises(ValueError):
        tdp.tdp_rope_freqs((1, 2))
    with pytest.raises(ValueError):
        tdp.tdp_rope_freqs((1, 2, 3), scaling="cubic")
    assert len(tdp.tdp_rope_table([], [])) == 0


def test_freqs(tdp):  # noqa: F811
    f, axis, scale = tdp.tdp_rope_freqs((5, 3, 0), base=500.0)
    assert np.allclose(f, [500.0 ** (-i / 5) for i in range(5)] + [500.0 ** (-i / 3) for i in range(3)], rtol=1e-14) and scale == 1
    assert axis.tolist() == [0] * 5 + [1] * 3
    assert np.allclose(tdp.tdp_rope_freqs((5, 3, 0), 500.0, "linear", 4.0)[0], f / 4, rtol=1e-15)
    g = tdp.tdp_rope_freqs((5, 3, 1), 500.0, "ntk", 4.0)[0]
    # the highest frequency stays, the lowest falls by the factor; one pair alone has nothing to fall
    assert g[0] == 1 and math.isclose(g[4], f[4] / 4, rel_tol=1e-13) and math.isclose(g[7], f[7] / 4, rel_tol=1e-13) and g[8] == 1
    y, _, scale = tdp.tdp_rope_freqs((64, 0, 0), 10000.0, "yarn", 16.0, 4096.0)
    assert np.allclose(y, ref.yarn(64, 10000.0, 16.0, 4096.0), rtol=1e-13) and math.isclose(scale, 0.1 * math.log(16) + 1, rel_tol=1e-6)
    assert y[0] == 1 and math.isclose(y[-1], 10000.0 ** (-63 / 64) / 16, rel_tol=1e-13)


def test_binding_refuses(tdp):  # noqa: F811
    import torch
    plan, x = _plan(tdp, "f32"), torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        tdp.tdp_rms_norm(plan, x, None, x)
    with pytest.raises(TypeError):
        tdp.tdp_rms_norm(plan, [1.0], None, x)
    with pytest.raises(ValueError):
        tdp.tdp_rms_norm(plan, torch.zeros(()), None, x)
    with pytest.raises(ValueError):
        tdp.tdp_quant8(plan, torch.zeros(4, 0), x, x)
    with pytest.raises(ValueError, match="rows of 32"):
        tdp.tdp_matmul8(plan, x, x, torch.zeros(8, 32), x, x)
    with pytest.raises(ValueError, match="rows must be"):
        tdp.tdp_rope(plan, x, x, torch.zeros(4, dtype=torch.int64), x)
    heads = torch.zeros(plan.total_tile_tokens, 2, 64)
    for other in (heads, heads.to_sparse(), heads.to("meta")):
        with pytest.raises(ValueError, match="CUDA"):
            tdp.tdp_rope(plan, other, x, torch.zeros(4, dtype=torch.int64), other)
    with pytest.raises(TypeError):
        tdp.tdp_rope(plan, heads, x, torch.zeros(4, dtype=torch.int64), None)


def test_header_and_binding_agree(tdp):  # noqa: F811
    src = open(os.path.join(os.path.dirname(tdp.LIB_PATH), "..", "include", "tdp.h")).read()
    assert f"#define TDP_MAX_NORM_BYTES {tdp.TDP_MAX_NORM_BYTES}" in src and f"#define TDP_MAX_ROPE_DIM {tdp.TDP_MAX_ROPE_DIM}" in src
    assert "#define TDP_MAX_MATMUL8 (1 << 20)" in src and tdp.TDP_MAX_MATMUL8 == 1 << 20
    assert "#define TDP_MAX_MATMUL8_ROWS (1 << 30)" in src and tdp.TDP_MAX_MATMUL8_ROWS == 1 << 30
    assert "#define TDP_MAX_ROPE_HEADS (1 << 20)" in src and tdp.TDP_MAX_ROPE_HEADS == 1 << 20
    assert ctypes.sizeof(tdp._Rope) == 6 * 4 + 4 * 8


@no_gpu_only
def test_outputs_in_one_place_refused(tdp):  # noqa: F811
    """Outputs on top of one another, or over a part of what others still read; 4 rows of 64 bf16 are 512 bytes, 256 in 8 bits."""
    lib, plan = tdp._lib, _plan(tdp)
    far = {n: (i + 2) << 16 for i, n in enumerate(("x", "res", "w", "h", "y", "rstd", "y8", "ys", "x8", "xs"))}

    def fwd(**kw):
        return lib.tdp_rms_norm(plan.handle, 4, 64, 1e-5, *(far | {k: far.get(v[0], 0) + v[1] for k, v in kw.items()}).values(), None)
    ok = (0, 6)             # launched, as far as that goes without a GPU
    assert fwd() in ok
    for a, b in (("h", "x"), ("h", "res"), ("y", "x"), ("y", "res")):
        assert fwd(**{a: (b, 0)}) in ok and fwd(**{a: (b, 16)}) == 1 and fwd(**{a: (b, -496)}) == 1 and fwd(**{a: (b, 512)}) in ok
    for a in ("y8", "x8"):
        for b in ("x", "res", "h", "y"):
            assert fwd(**{a: (b, 0)}) == 1 and fwd(**{a: (b, 496)}) == 1 and fwd(**{a: (b, 512)}) in ok and fwd(**{a: (b, -256)}) in ok
    assert fwd(y8=("x8", 0)) == 1 and fwd(y8=("x8", 240)) == 1 and fwd(y8=("x8", 256)) in ok and fwd(h=("y", 16)) == 1 and fwd(h=("y", 0)) == 1
    for a, b in (("rstd", "ys"), ("rstd", "xs"), ("ys", "xs")):
        assert fwd(**{a: (b, 0)}) == 1 and fwd(**{a: (b, 12)}) == 1 and fwd(**{a: (b, 16)}) in ok
    X = 1 << 20
    assert lib.tdp_quant8(plan.handle, 4, 64, X, X, 4 * X, None) == 1 and lib.tdp_quant8(plan.handle, 4, 64, X, X + 496, 4 * X, None) == 1
    assert lib.tdp_quant8(plan.handle, 4, 64, X, X + 512, 4 * X, None) in ok

    def grad(dx, h=None, x8=None):
        return lib.tdp_rms_norm_grad(plan.handle, 4, 64, h, x8, x8 and 5 * X, 6 * X, None, 2 * X, 3 * X, dx, None, None, 0, None)
    assert all(grad(d, h=X) in ok for d in (X, 2 * X, 3 * X, 4 * X)) and all(grad(d + 16, h=X) == 1 for d in (X, 2 * X, 3 * X))
    assert grad(X, x8=X) == 1 and grad(X - 496, x8=X) == 1 and grad(X - 512, x8=X) in ok

    def mm(out, res=None):
        return lib.tdp_matmul8(plan.handle, 4, 64, 64, X, 5 * X, 2 * X, 6 * X, None, res, out, None)
    assert mm(3 * X) in ok and mm(X) == 1 and mm(X + 240) == 1 and mm(2 * X + 4080) == 1 and mm(2 * X + 4096) in ok
    assert mm(3 * X, 3 * X) in ok and mm(3 * X, 3 * X + 16) == 1


def test_rows_of_another_shape_refused(tdp):  # noqa: F811
    """As many values in another order are not taken as they lie; flat ones, and dimensions that a row falls into, are."""
    import torch
    x = torch.zeros(8, 64)
    for bad in (torch.zeros(64, 8), torch.zeros(16, 32), torch.zeros(2, 2, 128)):
        with pytest.raises(ValueError, match="rows of 64"):
            tdp._ends(bad, "res", 64)
    for good in (x, x.view(-1), x.view(2, 4, 64), x.view(8, 4, 16), x.view(1, 8, 64), x.view(8, 64, 1)):
        tdp._ends(good, "res", 64)


def test_parts_of_a_pair_are_refused(tdp):  # noqa: F811
    for pairs in ((6.5, 5, 5), (6, 5, 0.5), np.array([6, 5, 5.25], np.float32)):
        with pytest.raises(ValueError, match="whole number"):
            tdp.tdp_rope_freqs(pairs)
    for pairs in (np.array([6, 5, 5], np.uint8), (6.0, 5, 5)):
        assert len(tdp.tdp_rope_freqs(pairs)[0]) == 16
