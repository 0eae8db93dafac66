"""The norm and the rotary positions under autograd, on the CPU: plain torch stands in for the library's calls, which like them
fill buffers that autograd does not see."""
import pytest

torch = pytest.importorskip("torch")

from test_abi_host import tdp  # noqa: E402,F401  (fixture)

R, C, H, D = 6, 16, 2, 8


def _norm(x, w, res, eps=1e-6):
    h = x if res is None else x + res
    return h, h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * (1 if w is None else w)


def _turn(x, back=False):
    """By one radian more a row."""
    t = torch.arange(x.shape[0], dtype=x.dtype)[:, None, None] * (-1 if back else 1)
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat((a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()), -1)


@pytest.fixture
def block(tdp, monkeypatch):  # noqa: F811
    from blend_tdp_tile_gb300 import block as b
    seen = []

    def aligned(*ts):
        for t in ts:
            if t is not None and (not t.is_contiguous() or t.data_ptr() % 16):
                raise ValueError("not 16-byte aligned")

    def rms_norm(plan, x, w, y=None, res=None, h=None, rstd=None, y8=None, y8_scale=None, x8=None, x8_scale=None, eps=1e-6):
        aligned(x, y, res, h, w)
        s, out = _norm(x, w, res, eps)
        y.copy_(out)
        rstd.copy_((s.square().mean(-1) + eps).rsqrt())
        if h is not None:
            h.copy_(s)
        if x8 is not None:
            x8_scale.fill_(1 / 64)
            x8.copy_((s * rstd[:, None] * 64).to(torch.float8_e4m3fn))

    def rms_norm_grad(plan, dy, dx, w, rstd, h=None, x8=None, x8_scale=None, dh=None, dw=None):
        aligned(dy, dx, dh)
        assert (h is None) != (x8 is None)
        seen.append("h" if x8 is None else "x8")
        u = h * rstd[:, None] if x8 is None else x8.float() * x8_scale[:, None]
        g = dy if w is None else dy * w
        dx.copy_(rstd[:, None] * (g - u * (g * u).mean(-1, keepdim=True)) + (0 if dh is None else dh))
        if dw is not None:
            dw.copy_((dy * u).sum(0))

    def rope(plan, x, Q, table, out, layout="half", at="middle", scale=1.0):
        if x.data_ptr() % 16 or any(s % 4 for s in x.stride()[:2]) or x.stride(-1) != 1:
            raise ValueError("not 16-byte aligned")
        out.copy_(_turn(x))

    def rope_grad(plan, x, Q, table, out, layout="half", at="middle", scale=1.0):
        if x.data_ptr() % 16 or any(s % 4 for s in x.stride()[:2]) or x.stride(-1) != 1:
            raise ValueError("not 16-byte aligned")
        out.copy_(_turn(x, True))

    for f in (rms_norm, rms_norm_grad, rope, rope_grad):
        monkeypatch.setattr(b, "tdp_" + f.__name__, f)
    b.seen = seen
    return b


def _calls(b):
    torch.manual_seed(0)
    w, res, Q, t = torch.randn(C), torch.randn(R, C), torch.zeros(6 * R, dtype=torch.int32), torch.zeros(D // 2, dtype=torch.int64)
    return {"rms_norm": (lambda x: b.rms_norm(None, x, w), torch.randn(R, C).requires_grad_()),
            "residual": (lambda x: torch.cat(b.rms_norm(None, x, w, res)), torch.randn(R, C).requires_grad_()),
            "rope": (lambda x: b.rope(None, x, Q, t), torch.randn(R, H, D).requires_grad_())}


@pytest.mark.parametrize("name", ["rms_norm", "residual", "rope"])
def test_first_derivatives(block, name):
    f, x = _calls(block)[name]
    y = f(x)
    w = torch.randn_like(y)
    got, = torch.autograd.grad((y * w).sum(), x)
    u, h = torch.randn_like(x), 2.0 ** -6
    with torch.no_grad():
        fd = float(((f(x + h * u).double() - f(x - h * u).double()) * w).sum()) / (2 * h)
    assert abs(fd - float((got * u).sum())) < 1e-2 * float((got * u).abs().sum())


@pytest.mark.parametrize("name", ["rms_norm", "residual", "rope"])
def test_second_derivatives_are_refused(block, name):
    f, x = _calls(block)[name]
    g, = torch.autograd.grad(f(x).pow(2).sum() + (x ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.pow(2).sum().backward()


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("used", ["y", "h", "both"])
def test_either_output_of_the_residual_norm(block, keep8, used):
    """x, res and w against plain torch, whichever outputs the loss reads; the checkpoint is off by e4m3's 2^-4."""
    torch.manual_seed(1)
    leaves = [torch.randn(R, C, requires_grad=True), torch.randn(C, requires_grad=True), torch.randn(R, C, requires_grad=True)]
    wy, wh = torch.randn(R, C), torch.randn(R, C)

    def loss(y, h):
        return ((y * wy).sum() if used != "h" else 0) + ((h * wh).sum() if used != "y" else 0)
    x, w, res = leaves
    got = torch.autograd.grad(loss(*block.rms_norm(None, x, w, res, keep8=keep8)), leaves, allow_unused=True)
    want = torch.autograd.grad(loss(*reversed(_norm(x, w, res))), leaves, allow_unused=True)
    assert block.seen == ([] if used == "h" else ["x8" if keep8 else "h"])
    for a, b in zip(got, want):
        if b is None:
            assert a is None or float(a.abs().max()) == 0
        else:
            assert float((a - b).abs().max()) < (0.3 if keep8 else 1e-4) * float(b.abs().max())


def test_a_stream_changed_before_backward_is_refused(block):
    x = torch.randn(R, C)
    w = torch.randn(C, requires_grad=True)
    y = block.rms_norm(None, x, w)
    x.zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = block.rms_norm(None, x, w, keep8=True)       # the checkpoint is its own
    x.fill_(1)
    y.sum().backward()


def test_positions_changed_before_backward_are_refused(block):
    Q, x = torch.zeros(6 * R, dtype=torch.int32), torch.randn(R, H, D, requires_grad=True)
    y = block.rope(None, x, Q, torch.zeros(D // 2, dtype=torch.int64))
    Q += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("name", ["rms_norm", "rope"])
def test_slices_at_odd_offsets(block, name, offset):
    f, x = _calls(block)[name]
    w = torch.randn(offset + x.numel())
    y = torch.cat([torch.zeros(offset, requires_grad=True) * 1, f(x).reshape(-1)])
    got, = torch.autograd.grad((y * w).sum(), x)
    want, = torch.autograd.grad((f(x).reshape(-1) * w[offset:].clone()).sum(), x)
    assert torch.equal(got, want)
    if name == "rms_norm":          # the weight too
        w1 = torch.cat([torch.zeros(offset), torch.ones(C)])[offset:]
        assert torch.equal(block.rms_norm(None, x.detach(), w1), block.rms_norm(None, x.detach(), w1.clone()))
    buf = torch.cat([torch.zeros(offset), x.detach().reshape(-1)])
    assert torch.equal(f(buf[offset:].view(x.shape)), f(x.detach()))


def test_layers_in_8_bits_refuse_gradients(block):
    lin = block.Linear8.__new__(block.Linear8)
    torch.nn.Module.__init__(lin)
    with pytest.raises(RuntimeError, match="no gradient"):
        lin(None, torch.randn(R, C, requires_grad=True))


class _BfPlan:
    esize = 2


@pytest.fixture
def block8(block, monkeypatch):
    """Plain products in 8 bits, which take what the library's take."""
    def quant8(plan, x, x8, x8_scale):
        assert x.dtype == torch.bfloat16
        x8_scale.copy_(x.float().abs().amax(-1).reshape(-1) / 448)
        x8.copy_((x.float() / x8_scale.view(*x.shape[:-1], 1)).to(torch.float8_e4m3fn))

    def matmul8(plan, x8, x8_scale, w8, w8_scale, out, bias=None, res=None):
        if w8.dtype not in (torch.uint8, torch.float8_e4m3fn) or w8_scale.dtype != torch.float32 or any(t is not None and t.dtype != torch.bfloat16 for t in (bias, res)):
            raise ValueError("dtype")
        y = (x8.float() * x8_scale.view(*x8.shape[:-1], 1)) @ (w8.view(torch.float8_e4m3fn).float() * w8_scale[:, None]).T
        out.copy_(y + (0 if bias is None else bias.float()) + (0 if res is None else res.float()))
    monkeypatch.setattr(block, "tdp_quant8", quant8)
    monkeypatch.setattr(block, "tdp_matmul8", matmul8)
    return block


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("change", [lambda m: m.to(torch.bfloat16), lambda m: m.bfloat16().float(), lambda m: m.half().double(), lambda m: m.float()])
def test_layers_in_8_bits_outlive_a_change_of_dtype(block8, bias, change):
    """Weights, scales and bias are what they were made as, whatever the module around them becomes."""
    torch.manual_seed(2)
    full = torch.nn.Linear(C, 24, bias=bias, dtype=torch.bfloat16)
    lin, x = block8.Linear8(_BfPlan, full), torch.randn(R, C).bfloat16()
    with torch.no_grad():
        want = lin(_BfPlan, x)
        around = change(torch.nn.Sequential(lin))
        assert torch.equal(around[0](_BfPlan, x), want)
    assert [(k, v.dtype) for k, v in lin.state_dict().items()] == \
        [("w8", torch.uint8), ("scale", torch.float32)] + ([("bias", torch.bfloat16)] if bias else [])
    other = block8.Linear8(_BfPlan, torch.nn.Linear(C, 24, bias=bias, dtype=torch.bfloat16))
    other.load_state_dict(lin.state_dict())
    with torch.no_grad():
        assert torch.equal(other(_BfPlan, x), want)


def _rotary(b, seed):
    torch.manual_seed(seed)
    return b.RotaryBlock(C, 2, 1, 8, 24, (2, 1, 1), dtype=torch.bfloat16, device="cpu")


def test_a_served_block_s_state_loads(block8):
    """Into a block that is not served in 8 bits, its weights; into one that is, those in 8 bits too."""
    served, fresh, other = _rotary(block8, 1).to_8bit(_BfPlan), _rotary(block8, 2), _rotary(block8, 3).to_8bit(_BfPlan)
    state = served.state_dict()
    fresh.load_state_dict(state)
    assert all(torch.equal(v, state[k]) for k, v in fresh.state_dict().items()) and fresh.in8 is None
    outer = torch.nn.ModuleDict({"a": _rotary(block8, 4)})
    outer.load_state_dict({"a." + k: v for k, v in state.items()})
    assert torch.equal(outer["a"].to_q.weight, served.to_q.weight)
    other.load_state_dict(state)
    for n, lin in other.in8.items():
        assert torch.equal(lin.w8, served.in8[n].w8) and torch.equal(lin.scale, served.in8[n].scale)
    with pytest.raises(RuntimeError, match="in8"):          # weights of another block beside 8-bit ones of this
        other.load_state_dict(fresh.state_dict())
    with pytest.raises(RuntimeError, match="other"):
        fresh.load_state_dict(state | {"other": torch.zeros(1)})


def test_the_gradient_takes_the_forward_s_scale(block, monkeypatch):
    """A factor in a tensor that changes between the two."""
    seen = []
    for name in ("tdp_rope", "tdp_rope_grad"):
        monkeypatch.setattr(block, name, lambda plan, x, Q, table, out, layout, at, scale: (seen.append(float(scale)), out.copy_(x)))
    scale, x = torch.tensor(1.5), torch.randn(R, H, D, requires_grad=True)
    y = block.rope(None, x, torch.zeros(6 * R, dtype=torch.int32), torch.zeros(D // 2, dtype=torch.int64), scale=scale)
    scale += 1
    y.sum().backward()
    assert seen == [1.5, 1.5]
