"""Masked cross attention whose lists of kept state tiles change from call to call at one address, with nothing between the
calls that waits for them."""
import threading

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


def _problem(tdp, seed, per_tile, D=64, S=700):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    plan = tdp.tdp_plan_create(2, 2, 9, 14, 8, "bf16", (1, 2, 2), (0, 2, 3))
    R, H, K = plan.B * plan.total_tile_tokens, 4, 2
    t = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    shape = (plan.n_tiles, plan.B, S) if per_tile else (plan.B, S)
    masks = []
    for keep, first in ((0.9, 0), (0.3, 384), (0.02, 500)):        # lists of six, three and two tiles
        m = torch.rand(shape, generator=g, device="cuda") < keep
        m[..., :first] = False
        masks.append(m)
    return plan, t(R, H, D), t(2, S, K, D), t(2, S, K, D), t(R, H, D), masks


def _call(tdp, plan, q, k, v, dout, mask, ws=None):
    import torch
    r = [torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]
    tdp.tdp_cross_attn(plan, q, k, v, mask, r[0], r[1], ws=ws)
    tdp.tdp_cross_attn_grad(plan, q, k, v, mask, r[0], r[1], dout, r[2], r[3], r[4], ws=ws)
    return r


def _same(a, b):
    import torch
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def _alone(tdp, plan, q, k, v, dout, masks):
    """Each mask's results from a workspace of its own, waited for."""
    import torch
    want = []
    for m in masks:
        n = max(tdp.tdp_cross_attn_workspace(plan, q, k, v, m, grad=g) for g in (False, True))
        want.append(_call(tdp, plan, q, k, v, dout, m, torch.zeros(n, dtype=torch.uint8, device="cuda")))
        torch.cuda.synchronize()
    return want


@pytest.mark.parametrize("per_tile", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_masks_in_turn(tdp, per_tile, D):
    import torch
    plan, q, k, v, dout, masks = _problem(tdp, 1, per_tile, D)
    want = _alone(tdp, plan, q, k, v, dout, masks)
    got = [_call(tdp, plan, q, k, v, dout, masks[i % 3]) for i in range(60)]
    torch.cuda.synchronize()
    assert all(_same(g, want[i % 3]) for i, g in enumerate(got))


def test_masks_in_turn_from_two_threads(tdp):
    """One plan, two threads, each on a stream of its own."""
    import torch
    plan, q, k, v, dout, masks = _problem(tdp, 2, True)
    want = _alone(tdp, plan, q, k, v, dout, masks)
    got = [[], []]

    def work(at):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[at] += [_call(tdp, plan, q, k, v, dout, masks[(i + at) % 3]) for i in range(40)]
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(at,)) for at in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for at in range(2):
        assert len(got[at]) == 40 and all(_same(g, want[(i + at) % 3]) for i, g in enumerate(got[at]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,S", [(1, 1000), (130, 130), (3000, 257), (700, 5000)])
def test_gradients_of_many_masked_tiles(tdp, D, T, S):
    """Rows of K to be zeroed in every tile, items of one state tile to forty: every tile of the ring is met by all its
    readers.  Each value of dq, dk and dv is a sum whose terms are rounded to bf16 twice and which is rounded once more: three
    independent errors of 2^-8 / sqrt(3) in the mean square at most, against 64 bits; delta, from an output that is
    rounded, adds a fourth."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + S)
    t = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    B, H, K = 3, 4, 2
    plan = tdp.tdp_plan_create(B, 1, 1, T, 8, "bf16", (1, 1, 1), (0, 0, 0))
    q, k, v, dout = t(B * T, H, D), t(B, S, K, D), t(B, S, K, D), t(B * T, H, D)
    mask = torch.rand(B, S, generator=g, device="cuda") < 0.6
    k[~mask], v[~mask] = float("nan"), float("inf")
    first = _call(tdp, plan, q, k, v, dout, mask)
    for _ in range(5):
        assert _same(_call(tdp, plan, q, k, v, dout, mask), first)
    for b in range(B):
        on, rows = mask[b], slice(b * T, (b + 1) * T)
        x, go = (a[rows].double().reshape(T, K, H // K, D) for a in (q, dout))
        kk, vv = k[b, on].double(), v[b, on].double()
        p = (torch.einsum("tkgd,skd->kgts", x, kk) * D ** -0.5).softmax(-1)
        dp = torch.einsum("tkgd,skd->kgts", go, vv)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * D ** -0.5
        want = (torch.einsum("kgts,skd->tkgd", ds, kk).reshape(T, H, D), torch.einsum("kgts,tkgd->skd", ds, x),
                torch.einsum("kgts,tkgd->skd", p, go))
        for name, got, w in zip(("dq", "dk", "dv"), (first[2][rows], first[3][b, on], first[4][b, on]), want):
            err = float((got.double() - w).norm() / w.norm())
            assert err < 2 * 2.0 ** -8 / 3 ** 0.5, (name, b, err)
    assert (first[3][~mask] == 0).all() and (first[4][~mask] == 0).all()


@pytest.mark.parametrize("S", [100, 300])
def test_a_forward_that_gave_up_shows_in_every_gradient(tdp, S):
    """What a forward that gave up leaves in a row, NaN in out and lse, is found in that row's dq and in the dk and dv of its
    item's states, and nowhere else."""
    import torch
    plan, q, k, v, dout, _ = _problem(tdp, 3, False, S=S)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    tdp.tdp_cross_attn(plan, q, k, v, None, out, lse)
    out[5, 1], lse[5, 1] = float("nan"), float("nan")          # item 0, key head 0
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    tdp.tdp_cross_attn_grad(plan, q, k, v, None, out, lse, dout, dq, dk, dv)
    lost = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    lost[5, 1] = True
    assert torch.equal(dq.isnan().all(-1), lost) and torch.equal(dq.isnan().any(-1), lost)
    for d in (dk, dv):
        assert d[0, :, 0].isnan().all() and not d[1].isnan().any() and not d[0, :, 1].isnan().any()
