"""The bounded waits of the paged attention in blocks of 128 rows: one that runs out (a copy that CTA 0 never asks for, on a working GPU: see
k3kda_test_arm_paged_wait_timeout) is reported through the workspace's status word; whatever else the kernel issued lands before it ends, and on
a workspace filled with zeros again the same call is as before."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import hybrid_linear_attention_rule_gb300 as K  # noqa: E402
from test_gpu_paged_attend import Case  # noqa: E402

TIMEOUT, TRIES = -6, 256


def _arm(tries):
    arm = K.load_library().k3kda_test_arm_paged_wait_timeout
    arm.argtypes, arm.restype = [ctypes.c_uint], None
    arm(tries)


@pytest.mark.parametrize("fmt", ["i4", "bf16"])
@pytest.mark.parametrize("total,new,heads,group", [([900] * 40, [64] * 40, 2, 4), ([5000] * 3, [200] * 3, 4, 1), ([30000], [130], 2, 2)], ids=str)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(total, new, heads, group, fmt):
    c = Case(total, new, heads, group, 128, 128, 64, fmt, (128, 0, "half"), seed=6)
    ws = K.paged_attend_workspace(c.cache, heads * group)
    want = c.run(ws=ws)
    assert K.k3kda_workspace_status(ws) == 0
    _arm(TRIES)
    c.run(ws=ws)
    assert K.k3kda_workspace_status(ws) == TIMEOUT
    assert K.k3kda_workspace_status(ws) == 0
    ws.zero_()
    for _ in range(2):
        assert torch.equal(c.run(ws=ws), want)
    assert K.k3kda_workspace_status(ws) == 0


def test_the_hook_is_taken_by_its_kernel_alone():
    """Armed for the blocks of rows, a call of few rows runs as ever; disarmed, so does the other."""
    few, many = Case([90], [1], 1, 1, 64, 64, 16, "i4"), Case([90], [90], 1, 1, 64, 64, 16, "i4")
    ws = K.paged_attend_workspace(few.cache, 1)
    a, b = few.run(ws=ws), many.run(ws=ws)
    _arm(TRIES)
    assert torch.equal(few.run(ws=ws), a) and K.k3kda_workspace_status(ws) == 0
    _arm(0)
    assert torch.equal(many.run(ws=ws), b) and K.k3kda_workspace_status(ws) == 0
