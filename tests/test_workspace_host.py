"""The small workspaces that a plan keeps, on the CPU: streams and allocations are stand-ins."""
import gc
import threading
import types
import weakref

import pytest

torch = pytest.importorskip("torch")

from test_abi_host import tdp  # noqa: E402,F401  (fixture)


@pytest.fixture
def streams(monkeypatch):
    """The current stream as (torch's id, raw handle); a stream that torch did not make has its handle as its id."""
    now = types.SimpleNamespace(id=0, handle=0, capturing=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: now.handle, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentStream", lambda dev: (now.id, dev, 1), raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now.capturing)

    def use(id, handle, capturing=False):
        now.id, now.handle, now.capturing = id, handle, capturing
    return use


@pytest.fixture
def take(tdp):  # noqa: F811
    plan = tdp.tdp_plan_create(1, 3, 8, 12, 16, "f32", (1, 2, 2), (0, 2, 2))
    like = types.SimpleNamespace(get_device=lambda: 0, device="cpu")
    return lambda need=1000: tdp._workspace(None, need, like, None, plan)


DEFAULT, POOLED, OTHER, EXTERNAL = (0, 0), (3, 0x7F00), (35, 0x7F80), (0x8000, 0x8000)


def test_one_a_stream(streams, take):
    first = {}
    for s in (DEFAULT, POOLED, OTHER):
        streams(*s)
        first[s] = take()
        assert first[s].numel() == 1000
    assert len({t.data_ptr() for t in first.values()}) == 3
    for s in (OTHER, DEFAULT, POOLED):
        streams(*s)
        assert take(500) is first[s]
    streams(*POOLED)
    assert take(2000).numel() == 2000 and take(1000).numel() == 2000


def test_streams_that_torch_did_not_make_keep_none(streams, take):
    """Such a stream may be destroyed with work on it, and another get its handle."""
    streams(*EXTERNAL)
    kept = weakref.ref(take())
    gc.collect()
    assert kept() is None


def test_captures_and_large_ones_keep_none(streams, take):
    streams(*POOLED, capturing=True)
    kept = weakref.ref(take())
    streams(*POOLED)
    large = weakref.ref(take((1 << 20) + 1))
    gc.collect()
    assert kept() is None and large() is None


def test_a_threads_go_with_it(streams, take):
    streams(*POOLED)
    mine, kept = take(), []

    def work():
        for s in (DEFAULT, POOLED):
            streams(*s)
            t = take()
            assert t is not mine and take() is t
            kept.append(weakref.ref(t))
    for _ in range(5):
        th = threading.Thread(target=work)
        th.start()
        th.join()
    gc.collect()
    assert len(kept) == 10 and all(k() is None for k in kept)
    streams(*POOLED)
    assert take() is mine
