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
