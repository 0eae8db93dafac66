"""The committed DRAM-traffic captures belong to the kernels as they are: bench.py gives no figure for a kernel whose sources
have changed since."""
import pytest

import bench


@pytest.mark.parametrize("call", sorted(bench.CALL_KERNELS))
@pytest.mark.parametrize("workload", ["tiny", "small", "medium", "temporal", "large"])
def test_traffic_is_there(call, workload):
    assert (bench.profiled_traffic(call, workload) or 0) > 0
