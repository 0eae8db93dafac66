"""tdp_dropout_add and tdp_dropout_grad: the mask word for word against Philox4x32-10 in numpy, the arithmetic against its one rounding."""
import numpy as np
import pytest

import block_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


def _plan(tdp, dtype):
    return tdp.tdp_plan_create(1, 1, 1, 1, 8, dtype, (1, 1, 1), (0, 0, 0))


def _rng(seed, offset):
    import torch
    return torch.from_numpy(np.array([seed, offset], np.uint64).view(np.int64)).cuda()


def test_generator_known_answers():
    """The published known-answer vectors of Philox4x32-10 (Random123): all zeros, all ones."""
    z = ref.philox_at([0], 0, 0)[0]
    assert [hex(int(w)) for w in z] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    m = 2 ** 64 - 1
    o = ref.philox_at([m], m, m)[0]
    assert [hex(int(w)) for w in o] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 4, 7, 8, 9, 1000, 4099, 1 << 20, 1234567])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_mask_and_values(tdp, dtype, n, p):
    import torch
    seed, offset = 0x123456789ABCDEF0 + n, (1 << 63) + 5
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(n)
    x, res = (torch.randn(n, generator=g).to(dt).cuda() for _ in range(2))
    keep = torch.from_numpy(ref.philox(n, seed, offset) >= np.uint64(round(p * 2 ** 32))).cuda()
    x[~keep] = float("nan")                    # a dropped element has no effect
    guard = torch.full((n + 64,), 3.0, dtype=dt, device="cuda")
    plan, rng = _plan(tdp, dtype), _rng(seed, offset)
    out = guard[:n]
    tdp.tdp_dropout_add(plan, x, res, p, rng, out)
    scaled = torch.where(keep, x.double() / (1 - p) if p < 1 else 0 * res.double(), 0)
    want = res.double() + scaled
    # fp32: the scale, the product and the sum, 2^-24 each of their terms; bf16 (8 significant bits) rounds once more, by 2^-8 at most
    tol = 3 * 2.0 ** -24 * (res.double().abs() + scaled.abs()) + (2.0 ** -8 * want.abs() * 1.01 if dtype == "bf16" else 0)
    assert ((out.double() - want).abs() <= tol).all()
    assert (guard[n:] == 3).all()
    dx = torch.full((n + 64,), 3.0, dtype=dt, device="cuda")
    tdp.tdp_dropout_grad(plan, x, p, rng, dx[:n])
    tol = 3 * 2.0 ** -24 * scaled.abs() + (2.0 ** -8 * scaled.abs() * 1.01 if dtype == "bf16" else 0)
    assert ((dx[:n].double() - scaled).abs() <= tol).all() and (dx[n:] == 3).all()
    assert ((dx[:n] != 0) <= keep).all()
    tdp.tdp_dropout_add(plan, x, None, p, rng, out)
    assert torch.equal(out, dx[:n])
    y = x.clone()                              # in place
    tdp.tdp_dropout_add(plan, y, None, p, rng, y)
    assert torch.equal(y, dx[:n])


def test_kept_share(tdp):
    import torch
    n, p = 1 << 24, 0.3
    x = torch.ones(n, device="cuda")
    out = torch.empty_like(x)
    tdp.tdp_dropout_add(_plan(tdp, "f32"), x, None, p, _rng(7, 0), out)
    kept = float((out != 0).double().mean())
    assert abs(kept - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5      # six standard deviations


def test_types_share_the_mask_and_offsets_change_it(tdp):
    import torch
    n = 100003
    x = torch.ones(n, device="cuda")
    a, b, c = torch.empty_like(x), torch.empty_like(x).bfloat16(), torch.empty_like(x)
    tdp.tdp_dropout_add(_plan(tdp, "f32"), x, None, 0.5, _rng(7, 1), a)
    tdp.tdp_dropout_add(_plan(tdp, "bf16"), x.bfloat16(), None, 0.5, _rng(7, 1), b)
    tdp.tdp_dropout_add(_plan(tdp, "f32"), x, None, 0.5, _rng(7, 2), c)
    assert torch.equal(a, b.float())
    assert 0.45 < float((a != c).double().mean()) < 0.55


def test_captured_graph_reads_the_offset(tdp):
    import torch
    n = 5000
    x, rng, plan = torch.ones(n, device="cuda"), _rng(3, 0), _plan(tdp, "f32")
    out = torch.empty_like(x)
    tdp.tdp_dropout_add(plan, x, None, 0.5, rng, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tdp.tdp_dropout_add(plan, x, None, 0.5, rng, out)
    for offset in (0, 1, 9):
        rng[1] = offset
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal((out != 0).cpu().numpy(), ref.philox(n, 3, offset) >= 2 ** 31)


def test_elements_past_32_bits(tdp):
    """Counters of 2^32 and more: the index's high word."""
    import torch
    n = (1 << 34) + 13
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    x[-64:] = 1
    tdp.tdp_dropout_add(_plan(tdp, "bf16"), x, None, 0.5, _rng(11, 3), x)
    i = np.arange(n - 64, n, dtype=np.uint64)
    words = ref.philox_at(i // np.uint64(4), 11, 3)[np.arange(64), (i % np.uint64(4)).astype(int)]
    assert np.array_equal(x[-64:].float().cpu().numpy(), np.where(words >= 2 ** 31, 2.0, 0.0))


def test_counters_past_32_bits(tdp):
    """2^34 elements and some: the counter's second word is no longer zero."""
    import torch
    n, seed, offset, p = (1 << 34) + (1 << 20) + 3, 0x123456789ABCDEF0, (1 << 63) + 5, 0.3
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    tdp.tdp_dropout_grad(_plan(tdp, "bf16"), x, p, _rng(seed, offset), x)
    for a, b in ((0, 4096), ((1 << 34) - 4096, (1 << 34) + 4096), ((n - 5000) // 4 * 4, n)):
        words = ref.philox_at(np.arange(a // 4, (b + 3) // 4), seed, offset).reshape(-1)[:b - a]
        assert np.array_equal(words >= np.uint64(round(p * 2 ** 32)), (x[a:b] != 0).cpu().numpy())
