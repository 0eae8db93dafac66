"""How the norm, the 8-bit products and the rotary positions are called: given streams, several threads, strides and broadcasts, a
first use inside a captured graph's warm-up, and the operators one after the other without a wait."""
import threading

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


def _state(tdp, seed, rows=700, C=512, N=384, dtype="bf16"):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    plan = tdp.tdp_plan_create(1, 1, 1, rows, 8, dtype, (1, 1, 1), (0, 0, 0))
    e = lambda *s, k=dt: torch.empty(s, dtype=k, device="cuda")  # noqa: E731
    f, b8 = torch.float32, torch.float8_e4m3fn
    s = dict(plan=plan, x=r(rows, C), res=r(rows, C), w=r(C), dy=r(rows, C), h=e(rows, C), y=e(rows, C), dx=e(rows, C), dw=e(C, k=f), rstd=e(rows, k=f),
             y8=e(rows, C, k=b8), ys=e(rows, k=f), w8=e(N, C, k=b8), ws=e(N, k=f), out=e(rows, N), turned=e(rows, N // 64, 64), back=e(rows, N // 64, 64),
             Q=torch.randint(0, 99, (6 * rows,), generator=g, device="cuda", dtype=torch.int32),
             table=tdp.tdp_rope_table(*tdp.tdp_rope_freqs((16, 8, 8))[:2]).cuda())
    tdp.tdp_quant8(plan, r(N, C), s["w8"], s["ws"])
    return s


def _chain(tdp, s, **kw):
    """Each call reads what the one before it wrote."""
    p = s["plan"]
    tdp.tdp_rms_norm(p, s["x"], s["w"], s["y"], res=s["res"], h=s["h"], rstd=s["rstd"], y8=s["y8"], y8_scale=s["ys"], **kw)
    tdp.tdp_matmul8(p, s["y8"], s["ys"], s["w8"], s["ws"], s["out"], **kw)
    tdp.tdp_rope(p, s["out"].view(s["turned"].shape), s["Q"], s["table"], s["turned"], **kw)
    tdp.tdp_rope_grad(p, s["turned"], s["Q"], s["table"], s["back"], **kw)
    tdp.tdp_rms_norm_grad(p, s["dy"], s["dx"], s["w"], s["rstd"], h=s["h"], dh=s["y"], dw=s["dw"], **kw)


OUT = ("h", "y", "rstd", "y8", "ys", "out", "turned", "back", "dx", "dw")


def _same(a, b):
    import torch
    for k in OUT:
        x, y = a[k], b[k]
        if x.dtype == torch.float8_e4m3fn:
            x, y = x.view(torch.uint8), y.view(torch.uint8)
        assert torch.equal(x, y), k


@pytest.mark.parametrize("rows", [9, 700, 30000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_given_streams(tdp, rows, dtype):
    import torch
    want, a, b = (_state(tdp, 5, rows, dtype=dtype) for _ in range(3))
    _chain(tdp, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    _chain(tdp, a, stream=side)
    _chain(tdp, b, stream=side.cuda_stream)         # a handle
    side.synchronize()
    _same(a, want)
    _same(b, want)


def test_threads(tdp):
    """Four threads, a plan and a stream each, and one plan that two of them share."""
    import torch
    states = [_state(tdp, i, 300 + 17 * i) for i in range(4)]
    want = [_state(tdp, i, 300 + 17 * i) for i in range(4)]
    for s in want:
        _chain(tdp, s)
    shared = _state(tdp, 2, 334)
    shared["plan"] = states[2]["plan"]
    states.append(shared)
    want.append(want[2])
    torch.cuda.synchronize()
    wrong = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    _chain(tdp, s)
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # a thread's error would go unseen
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(s,)) for s in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    for s, w in zip(states, want):
        _same(s, w)


def test_two_graphs_at_once(tdp):
    import torch
    a, b, want = _state(tdp, 1), _state(tdp, 1), _state(tdp, 1)
    _chain(tdp, want)
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _chain(tdp, s)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    _same(a, want)
    _same(b, want)


def test_broadcast_and_refused_strides(tdp):
    import torch
    s = _state(tdp, 3, 40)
    one = torch.randn(40, 1, 64, device="cuda").bfloat16()
    many = torch.empty(40, 6, 64, dtype=torch.bfloat16, device="cuda")
    tdp.tdp_rope(s["plan"], one.expand(40, 6, 64), s["Q"], s["table"], many)       # a head for all
    want = torch.empty_like(one)
    tdp.tdp_rope(s["plan"], one, s["Q"], s["table"], want)
    assert torch.equal(many, want.expand(40, 6, 64))
    with pytest.raises(tdp.TdpError):                                             # outputs on top of one another
        tdp.tdp_rope(s["plan"], many, s["Q"], s["table"], one.expand(40, 6, 64))
    for bad in (many[:, :, ::2], many.transpose(1, 2)[:, :, :6]):
        with pytest.raises(ValueError):
            tdp.tdp_rope(s["plan"], bad, s["Q"], s["table"], torch.empty_like(bad))
    # what is kept of a shape that was right says nothing of the next call's buffers
    buf = torch.empty(40 * 6 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="aligned"):
        tdp.tdp_rope(s["plan"], many, s["Q"], s["table"], buf[1:1 + many.numel()].view(many.shape))
    with pytest.raises(ValueError, match="dtype"):
        tdp.tdp_rope(s["plan"], many.float(), s["Q"], s["table"], many)
    with pytest.raises(ValueError, match="shape"):
        tdp.tdp_rope(s["plan"], many, s["Q"], s["table"], many[:, :5])
    with pytest.raises(ValueError, match="elements"):
        tdp.tdp_rope(s["plan"], many, s["Q"][:-1], s["table"], many)
    with pytest.raises(ValueError, match="layout"):
        tdp.tdp_rope(s["plan"], many, s["Q"], s["table"], many, layout="other")
    with pytest.raises(ValueError, match="contiguous"):
        tdp.tdp_rms_norm(s["plan"], s["x"][:, ::2], None, s["y"][:, ::2])
    with pytest.raises(ValueError, match="dtype"):
        tdp.tdp_matmul8(s["plan"], s["y8"].view(torch.float8_e5m2), s["ys"], s["w8"], s["ws"], s["out"])
    with pytest.raises(ValueError, match="elements"):
        tdp.tdp_matmul8(s["plan"], s["y8"], s["ys"][:-1], s["w8"], s["ws"], s["out"])
    with pytest.raises(tdp.TdpError):
        tdp.tdp_rms_norm(s["plan"], s["x"], None, s["y"], h=s["y"])


def test_rows_of_another_shape_are_refused(tdp):
    """As many values in another order; flat ones, and dimensions that a row falls into, give what rows give."""
    import torch
    s = _state(tdp, 4, 40)
    p, x, r, dy = s["plan"], s["x"], s["res"], s["dy"]
    rows, C = x.shape
    dt, rstd = x.dtype, torch.rand(rows, device="cuda")
    e = lambda *n, k=dt: torch.empty(n or (rows, C), dtype=k, device="cuda")  # noqa: E731
    ys, b8 = e(rows, k=torch.float32), torch.uint8
    calls = {"res": lambda t, o: tdp.tdp_rms_norm(p, x, None, o, res=t), "dh": lambda t, o: tdp.tdp_rms_norm_grad(p, dy, o, None, rstd, h=x, dh=t),
             "kept": lambda t, o: tdp.tdp_rms_norm_grad(p, dy, o, None, rstd, h=t)}
    for f in calls.values():
        want = e()
        f(r, want)
        for shape in ((rows * C,), (2, rows // 2, C), (rows, 8, C // 8)):
            got = e(*shape)
            f(r.view(shape), got)
            assert torch.equal(got.view(rows, C), want)
        for t in (r.view(C, rows), r.view(2 * rows, C // 2)):
            with pytest.raises(ValueError, match="rows of"):
                f(t, want)
            with pytest.raises(ValueError, match="rows of"):
                f(r, e(*t.shape))
    for f in (lambda t: tdp.tdp_rms_norm(p, x, None, None, h=t), lambda t: tdp.tdp_rms_norm(p, x, None, None, y8=t.view(b8)[..., ::2].contiguous(), y8_scale=ys),
              lambda t: tdp.tdp_quant8(p, x, t.view(b8)[..., ::2].contiguous(), ys)):
        f(e())
        with pytest.raises(ValueError, match="rows of"):
            f(e(C, rows))
    N = s["out"].shape[1]
    for f in (lambda t: tdp.tdp_matmul8(p, s["y8"], s["ys"], s["w8"], s["ws"], t), lambda t: tdp.tdp_matmul8(p, s["y8"], s["ys"], s["w8"], s["ws"], s["out"], res=t)):
        f(e(rows, N)), f(e(rows * N)), f(e(rows, N // 64, 64))
        with pytest.raises(ValueError, match="rows of"):
            f(e(N, rows))
