"""The gated delta rule's wait for a record that is being made, made to run out without a
fault: with the first record's flag withheld, its head's chains give up after their limit of
looks, record SSM_ERR_TIMEOUT in the workspace and finish; other heads are right, and so is the
next call."""
import time

import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests.test_gated_delta_gpu import F32, cuda, forward, inputs

pytestmark = pytest.mark.gpu

OK, TIMEOUT = 0, 7


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 40)])
def test_a_record_that_is_never_told_of(dk, dv):
    n, h = 8192, 8   # so many that records are made beside the chains
    c = cuda(inputs(1, n, h, h, dk, dv, seed=31))
    ws = torch.empty(binding.ssm_gated_delta_workspace_bytes(1, n, h, dk, dv), dtype=torch.uint8,
                     device="cuda")
    want = forward(c, out_dtype=F32, workspace=ws)
    assert binding.ssm_last_device_status(ws) == OK
    try:
        binding.ssm_debug_set_lookback(True, 2000)
        start = time.perf_counter()
        y, last = forward(c, out_dtype=F32, workspace=ws)
        status = binding.ssm_last_device_status(ws)
        elapsed = time.perf_counter() - start
    finally:
        binding.ssm_debug_set_lookback()
    assert status == TIMEOUT
    assert elapsed < 0.5, elapsed  # the shortened limit, no other wait behind it
    assert torch.equal(y[:, :, 1:], want[0][:, :, 1:]) and torch.equal(last[:, 1:], want[1][:, 1:])
    again = forward(c, out_dtype=F32, workspace=ws)
    assert binding.ssm_last_device_status(ws) == OK
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_a_limit_of_looks_alone_changes_nothing():
    c = cuda(inputs(1, 8192, 8, 8, 64, 64, seed=32))
    ws = torch.empty(binding.ssm_gated_delta_workspace_bytes(1, 8192, 8, 64, 64), dtype=torch.uint8,
                     device="cuda")
    want = forward(c, workspace=ws)
    try:
        binding.ssm_debug_set_lookback(False, 1 << 21)
        got = forward(c, workspace=ws)
        status = binding.ssm_last_device_status(ws)
    finally:
        binding.ssm_debug_set_lookback()
    assert status == OK and all(torch.equal(a, b) for a, b in zip(got, want))
