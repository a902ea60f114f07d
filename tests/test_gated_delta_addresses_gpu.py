"""Gated delta rule with tensors at any address that the entry points take: multiples of 16
bytes, of 32 or not.  The same kernels on the same values: bit-equal to tensors of their own."""
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests.test_gated_delta_gpu import BF16, F32, backward, cuda, forward, inputs

pytestmark = pytest.mark.gpu


def at(shape, dt, skip):
    """A tensor whose first element lies `skip` bytes behind a multiple of 256."""
    size = torch.Size(shape).numel()
    room = torch.full((size + 256,), 7.0, dtype=dt, device="cuda")
    first = skip // room.element_size()
    view = room[first:first + size].view(shape)
    assert view.data_ptr() % 256 == skip
    return view, room


def untouched(view, room):
    first = view.storage_offset()
    return (room[:first] == 7).all() and (room[first + view.numel():] == 7).all()


# widths whose rows are multiples of 32 bytes in bf16, and not; lengths in chunks and walked
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (16, 48), (72, 40)])
@pytest.mark.parametrize("n,h", [(7, 3), (130, 4), (70, 200)])
@pytest.mark.parametrize("skip", [16, 48, 32])
def test_outputs_behind_any_16_bytes(dk, dv, n, h, skip):
    groups = h // 2 if h % 2 == 0 else h
    c = cuda(inputs(1, n, h, groups, dk, dv, seed=dk + n))
    for dt in (BF16, F32):
        want_y, want_s = forward(c, out_dtype=dt)
        y, y_room = at(c["v"].shape, dt, skip)
        s, s_room = at(c["state"].shape, F32, skip)
        forward(c, out_dtype=dt, y=y, final_state=s)
        assert torch.equal(y, want_y) and torch.equal(s, want_s)
        assert untouched(y, y_room) and untouched(s, s_room)
        want = backward(c, grad_dtype=dt)
        out = {k: at(v.shape, v.dtype, skip) for k, v in want.items()}
        backward(c, grad_dtype=dt, out={k: v for k, (v, _) in out.items()})
        for k, (v, room) in out.items():
            assert torch.equal(v, want[k]) and untouched(v, room), k


@pytest.mark.parametrize("n", [6, 130])
def test_inputs_and_workspaces_behind_any_16_bytes(n):
    c = cuda(inputs(2, n, 4, 2, 64, 64, seed=n))
    want = forward(c), backward(c)
    moved = {}
    for k, t in c.items():
        moved[k], _ = at(t.shape, t.dtype, 16)
        moved[k].copy_(t)
    five = 2, n, 4, 64, 64
    sizes = (binding.ssm_gated_delta_workspace_bytes(*five),
             binding.ssm_gated_delta_bwd_workspace_bytes(*five) +
             binding.ssm_gated_delta_checkpoint_bytes(*five),
             binding.ssm_gated_delta_checkpoint_bytes(*five),
             binding.ssm_gated_delta_bwd_workspace_bytes(*five))
    ws = [torch.empty(s + 16, dtype=torch.uint8, device="cuda")[16:] for s in sizes]
    got = forward(moved, workspace=ws[0]), backward(moved, workspace=ws[1])
    assert all(torch.equal(a, b) for a, b in zip(want[0], got[0]))
    assert all(torch.equal(want[1][k], got[1][k]) for k in want[1])
    forward(moved, checkpoints=ws[2])
    got = backward(moved, checkpoints=ws[2], workspace=ws[3])
    assert all(torch.equal(want[1][k], got[k]) for k in want[1])
