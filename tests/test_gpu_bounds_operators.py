"""The tests of the expert selection, the routed layer and the adapters again on
the bounds-checked build (libmoe_bounds.so, MOE_LIBRARY=bounds), which records
every index read from data -- plans, tasks, rows, ranks, routings -- that leaves
its range in the status word; these tests check that word after their calls.
Each group is a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

GROUPS = {
    "selection": ["tests/test_gpu_gate.py", "-k", "layer_routed or route_gated or together or masked or groups"],
    "adapters": ["tests/test_gpu_adapter.py"],
    "adapter_widths": ["tests/test_gpu_adapter_sizes.py", "-k", "smallest"],
}


@pytest.mark.parametrize("group", list(GROUPS))
def test_on_the_bounds_checked_build(group):
    assert os.path.exists(os.path.join(ROOT, "expert_ffn_router_b200", "libmoe_bounds.so")), "libmoe_bounds.so is not built"
    env = dict(os.environ, MOE_LIBRARY="bounds")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider"] +
                       GROUPS[group], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert "passed" in r.stdout
