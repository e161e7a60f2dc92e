"""A bounded wait inside the tensor-core attention that runs out: error 2, a
clean return, and a context and a cache that the next call can use."""
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.test_gpu_tree_units import Units

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("D,group,T", [(128, 4, 8), (64, 8, 1), (128, 8, 6), (64, 8, 6), (128, 3, 64), (64, 5, 40)])
def test_a_wait_that_runs_out_is_reported(cuda, monkeypatch, D, group, T):
    """DSPARK_TEST_STALL_WAIT=1 makes the warp that issues the products wait,
    behind its first scores, for a barrier phase that nothing completes, with a
    short limit.  The other warps' waits run out behind it (2 s), copies and
    products under way are waited for, and the next call is clean."""
    s = Units(BF, D, 8, group, T, [700, 130, 0, 1000], 16, "causal", seed=T)
    a = dict(out=torch.zeros_like(s.q), lse=torch.zeros(4, T, 8 * group, device="cuda"),
             workspace=dspark.TreeWorkspace(4, T, 8 * group, 8, D))
    s.run(**a)
    s.check(a["out"], a["lse"])
    want = [a["out"].clone(), a["lse"].clone()]
    pool = s.c.pool.view(torch.int16).clone()
    monkeypatch.setenv("DSPARK_TEST_STALL_WAIT", "1")
    s.run(**a)
    torch.cuda.synchronize()
    assert dspark.read_device_error(s.c) == 2 and dspark.read_device_error(s.c) == 0
    monkeypatch.delenv("DSPARK_TEST_STALL_WAIT")
    s.run(**a)
    assert torch.equal(a["out"], want[0]) and torch.equal(a["lse"], want[1])
    assert dspark.read_device_error(s.c) == 0
    assert torch.equal(s.c.pool.view(torch.int16), pool)
