"""The small workspaces that a plan keeps: torch's streams have one each, other streams none."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tdp():
    import __graft_entry__
    __graft_entry__.build()
    import blend_tdp_tile_gb300
    return blend_tdp_tile_gb300


def test_streams_of_torch_and_of_others(tdp):
    import torch
    plan = tdp.tdp_plan_create(1, 3, 8, 12, 8, "f32", (1, 2, 2), (0, 2, 2))
    C, G = 64, 8
    x = torch.randn(plan.total_tile_tokens, C, device="cuda")

    def norm():
        y, mean, rstd = torch.empty_like(x), torch.empty(plan.n_tiles * G, device="cuda"), torch.empty(plan.n_tiles * G, device="cuda")
        tdp.tdp_group_norm(plan, x, G, None, None, y, mean, rstd)
        return y
    want = norm()
    torch.cuda.synchronize()
    kept = dict(plan.scratch.by_stream)
    assert list(kept) == [(0, 0)]
    # a stream that torch did not make
    rt, handle = ctypes.CDLL("libcudart.so.13"), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(handle), 1) == 0
    try:
        with torch.cuda.stream(torch.cuda.ExternalStream(handle.value)):
            got = [norm() for _ in range(6)]
            torch.cuda.current_stream().synchronize()
        assert list(plan.scratch.by_stream) == [(0, 0)]
    finally:
        torch.cuda.synchronize()
        rt.cudaStreamDestroy(handle)
    # streams that it did make
    for s in (torch.cuda.default_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            got.append(norm())
            ws = plan.scratch.by_stream[0, s.stream_id]
            got.append(norm())
            assert plan.scratch.by_stream[0, s.stream_id] is ws
        s.synchronize()
    assert plan.scratch.by_stream[0, 0] is kept[0, 0]
    assert all(torch.equal(y, want) for y in got)
