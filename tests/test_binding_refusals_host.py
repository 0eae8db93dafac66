"""Tensors that have no memory to point at are refused as any other that is not on the GPU."""
import pytest

torch = pytest.importorskip("torch")

from test_abi_host import tdp  # noqa: E402,F401  (fixture)


@pytest.mark.parametrize("kind", ["sparse", "meta", "plain"])
def test_not_a_cuda_tensor(tdp, kind):  # noqa: F811
    plan = tdp.tdp_plan_create(1, 3, 8, 12, 16, "f32", (1, 2, 2), (0, 2, 2))
    x = {"sparse": lambda: torch.zeros(4, 4).to_sparse(), "meta": lambda: torch.zeros(8, device="meta"),
         "plain": lambda: torch.zeros(8)}[kind]()
    for call in (lambda: tdp.tdp_blend(plan, x, x), lambda: tdp._ptr(x, "x", x.numel(), (torch.float32,), 16)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
