"""The block's operators under autograd, on the CPU: plain torch stands in for the library's calls, which like them fill
buffers that autograd does not see."""
import pytest

torch = pytest.importorskip("torch")

from test_abi_host import tdp  # noqa: E402,F401  (fixture)


def _gn(x, groups, gamma, beta, eps, act):
    h = torch.nn.functional.group_norm(x.t()[None], groups, gamma, beta, eps)[0].t()
    return torch.nn.functional.silu(h) if act == "silu" else h


def _attn(q, k, v, mask):
    s = torch.einsum("thd,shd->hts", q, k[0]) * q.shape[-1] ** -0.5
    s = s if mask is None else s.masked_fill(~mask[0], float("-inf"))
    return torch.einsum("hts,shd->thd", s.softmax(-1), v[0]), s.logsumexp(-1).t()


@pytest.fixture
def block(tdp, monkeypatch):  # noqa: F811
    from blend_tdp_tile_gb300 import block as b

    def aligned(*ts):
        for t in ts:
            if not t.is_contiguous() or t.data_ptr() % 16:
                raise ValueError("not 16-byte aligned")

    def group_norm(plan, x, groups, gamma, beta, y, mean, rstd, eps=1e-5, act="none"):
        aligned(x, y)
        y.copy_(_gn(x, groups, gamma, beta, eps, act))

    def group_norm_grad(plan, x, groups, gamma, beta, mean, rstd, dy, dx, dgamma=None, dbeta=None, act="none"):
        aligned(x, dy, dx)
        with torch.enable_grad():
            ins = [t.detach().requires_grad_() for t in (x, gamma, beta)]
            got = torch.autograd.grad(_gn(ins[0], groups, ins[1], ins[2], 1e-5, act), ins, dy)
        for to, g in zip((dx, dgamma, dbeta), got):
            to.copy_(g)

    def cross_attn(plan, q, k, v, mask, out, lse=None, scale=None):
        o, l = _attn(q, k, v, mask)
        out.copy_(o)
        lse.copy_(l)

    def cross_attn_grad(plan, q, k, v, mask, out, lse, dout, dq, dk, dv, scale=None):
        aligned(out, dout, dq, dk, dv)
        with torch.enable_grad():
            ins = [t.detach().requires_grad_() for t in (q, k, v)]
            got = torch.autograd.grad(_attn(*ins, mask)[0], ins, dout)
        for to, g in zip((dq, dk, dv), got):
            to.copy_(g)

    def dropout_add(plan, x, res, p, rng, out):
        aligned(x, out, *(() if res is None else (res,)))
        out.copy_(x / (1 - p) + (0 if res is None else res))

    def dropout_grad(plan, dout, p, rng, dx):
        aligned(dout, dx)
        dx.copy_(dout / (1 - p))

    for f in (group_norm, group_norm_grad, cross_attn, cross_attn_grad, dropout_add, dropout_grad):
        monkeypatch.setattr(b, "tdp_" + f.__name__, f)
    return b


class _Plan:
    n_tiles = B = 1


T, C, S, H, D = 6, 8, 5, 2, 4


def _calls(b):
    """name -> (function of one leaf, the leaf)."""
    torch.manual_seed(0)
    r = lambda *s: torch.randn(s)  # noqa: E731
    gamma, beta, k, v, res, rng = r(C), r(C), r(1, S, H, D), r(1, S, H, D), r(T, C), torch.zeros(2, dtype=torch.int64)
    return {"group_norm": (lambda x: b.group_norm(_Plan, x, 2, gamma, beta), r(T, C).requires_grad_()),
            "cross_attn": (lambda q: b.cross_attn(_Plan, q, k, v), r(T, H, D).requires_grad_()),
            "dropout_add": (lambda x: b.dropout_add(_Plan, x, res, 0.5, rng) ** 2, r(T, C).requires_grad_())}


@pytest.mark.parametrize("name", ["group_norm", "cross_attn", "dropout_add"])
def test_second_derivatives_are_refused(block, name):
    """A gradient penalty's derivative would lack the operator's own second derivative: it is an error, not a number."""
    f, x = _calls(block)[name]
    g, = torch.autograd.grad((f(x) + x ** 2).pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.pow(2).sum().backward()


@pytest.mark.parametrize("name", ["group_norm", "cross_attn", "dropout_add"])
def test_first_derivatives(block, name):
    f, x = _calls(block)[name]
    w = torch.randn_like(x)
    got, = torch.autograd.grad((f(x) * w).sum(), x)
    u, h = torch.randn_like(x), 2.0 ** -6
    with torch.no_grad():
        fd = float(((f(x + h * u).double() - f(x - h * u).double()) * w).sum()) / (2 * h)
    assert abs(fd - float((got * u).sum())) < 1e-2 * float((got * u).abs().sum())


def test_a_mask_refilled_before_backward_is_refused(block):
    """lse belongs to the forward's mask; gradients under another one would be of no function."""
    q, k, v = torch.randn(T, H, D, requires_grad=True), torch.randn(1, S, H, D), torch.randn(1, S, H, D)
    mask = torch.tensor([[True, True, False, True, False]])
    block.cross_attn(_Plan, q, k, v, mask).sum().backward()
    assert q.grad is not None
    out = block.cross_attn(_Plan, q, k, v, mask)
    mask.fill_(True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("name", ["group_norm", "cross_attn", "dropout_add"])
def test_gradients_that_are_slices_at_odd_offsets(block, name, offset):
    """A cat's gradient is slices of one buffer: contiguous, and wherever they happen to start."""
    f, x = _calls(block)[name]
    w = torch.randn(offset + x.numel())
    y = torch.cat([torch.zeros(offset, requires_grad=True) * 1, f(x).reshape(-1)])
    got, = torch.autograd.grad((y * w).sum(), x)
    want, = torch.autograd.grad((f(x).reshape(-1) * w[offset:].clone()).sum(), x)
    assert torch.equal(got, want)


def test_inputs_that_are_slices_at_odd_offsets(block):
    """What the functions copy where it is not contiguous they copy where it is not aligned."""
    rng = torch.zeros(2, dtype=torch.int64)
    buf = torch.randn(2 * T * C + 2)
    x, res = buf[1:1 + T * C].view(T, C), buf[1 + T * C:1 + 2 * T * C].view(T, C)
    assert torch.equal(block.dropout_add(_Plan, x, res, 0.5, rng), block.dropout_add(_Plan, x.clone(), res.clone(), 0.5, rng))
    gamma, beta = torch.randn(C), torch.randn(C)
    assert torch.equal(block.group_norm(_Plan, x, 2, gamma, beta), block.group_norm(_Plan, x.clone(), 2, gamma, beta))
