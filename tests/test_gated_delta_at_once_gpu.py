"""Gated delta rule over sequences long enough, of heads few enough, that records are made
beside the chains that follow them: the same records and chains as one after the other."""
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests.test_gated_delta_gpu import BF16, F32, FWD, cuda, forward, inputs, off, reference

pytestmark = pytest.mark.gpu


# odd ends and widths; shared keys; several sequences; the most heads that fit beside makers
@pytest.mark.parametrize("b,n,h,groups,dk,dv", [(1, 8190, 8, 8, 128, 128), (1, 5000, 12, 4, 72, 40), (2, 6001, 6, 3, 64, 200),
                                                (3, 4100, 4, 4, 16, 8), (1, 3000, 18, 18, 128, 128)])
def test_at_once(b, n, h, groups, dk, dv):
    t = inputs(b, n, h, groups, dk, dv, seed=n, restart=0.002)
    c = cuda(t)
    ws = torch.empty(binding.ssm_gated_delta_workspace_bytes(b, n, h, dk, dv), dtype=torch.uint8, device="cuda")
    y_ref, last_ref = reference(t)
    y, last = forward(c, out_dtype=F32, workspace=ws)
    assert binding.ssm_last_device_status(ws) == 0
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    yb, lastb = forward(c, out_dtype=BF16, workspace=ws)
    assert torch.equal(yb, y.to(BF16)) and torch.equal(lastb, last)
    for _ in range(10):
        again = forward(c, out_dtype=F32, workspace=ws)
        assert binding.ssm_last_device_status(ws) == 0
        assert torch.equal(again[0], y) and torch.equal(again[1], last)


def test_two_at_once_and_captured():
    a, b = (cuda(inputs(1, 6000, 8, 8, 128, 128, seed=s)) for s in (41, 42))
    want = [forward(a), forward(b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, (c, s) in enumerate(zip((a, b), streams)):
            outs[i].append(forward(c, stream=s))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = forward(a)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    outs[0].append(captured)
    for got, ref in zip(outs, want):
        for y, last in got:
            assert torch.equal(y, ref[0]) and torch.equal(last, ref[1])
