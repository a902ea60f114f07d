"""Tensors of more than 2^31 elements through the norms of heads and the gated delta rule: what
lies at their ends against the plain form, or against the same heads in a call of their own.
Tolerances as in the operators' own tests."""
import numpy as np
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests import plain64_heads as H
from tests.helpers import to64
from tests.test_gated_delta_gpu import BWD, GATES, ROUND

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _randn(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape, dtype=BF16: torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def near(got, ref, tol):
    assert np.linalg.norm(to64(got) - ref) < tol * np.linalg.norm(ref)


# angles held; neighbouring columns; heads of an odd width, ranges of a projection
@pytest.mark.parametrize("dim,rot,interleaved,extra", [(128, 128, False, 0), (128, 64, True, 0), (72, 20, False, 8)])
def test_qk_norm(dim, rot, interleaved, extra):
    qheads, kheads = 48, 16
    n = (2 ** 31 + 2 ** 27) // (qheads * dim)
    randn = _randn(1)
    wide = randn(1, n, (qheads + kheads) * dim + extra)
    q = wide[..., :qheads * dim].unflatten(-1, (qheads, dim))
    k = wide[..., qheads * dim:(qheads + kheads) * dim].unflatten(-1, (kheads, dim))
    w = 1 + 0.1 * randn(dim, dtype=F32)
    positions = torch.arange(n, device="cuda")[None] + (1 << 20)
    freq = 10000.0 ** (-2 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    a = dict(q_weight=w, positions=positions, inv_freq=freq, eps=EPS, interleaved=interleaved)
    q_out, k_out = binding.ssm_qk_norm_rope_fwd(q, k, **a)
    g = binding.ssm_qk_norm_rope_bwd(q_out, k_out, q, k, **a)
    edges = (0, 2 ** 31 // (qheads * dim) - 4, 2 ** 31 // wide.shape[2] - 4, n - 8)
    for at in (slice(i, i + 8) for i in edges):
        phase = H.angles(positions[:, at].cpu().numpy(), to64(freq))
        for x, wt, y, dx in ((q, w, q_out, g["dq"]), (k, None, k_out, g["dk"])):
            x64, w64 = to64(x[:, at]), None if wt is None else to64(wt)
            near(y[:, at], H.qk_fwd(x64, w64, phase, rot, EPS, interleaved), 2.5e-3)
            near(dx[:, at], H.qk_bwd(x64, w64, phase, rot, EPS, to64(y[:, at]), interleaved)[0], 2.5e-3)
    # y turned back is n w: dw is the sum of n^2 w, but for y's rounding to bf16
    dw = torch.zeros(dim, dtype=torch.float64, device="cuda")
    for t in range(0, n, 16384):
        x = q[0, t:t + 16384].double()
        dw += (x.square() / (x.square().mean(-1, keepdim=True) + EPS)).sum((0, 1)) * w.double()
    near(g["dq_weight"], to64(dw), 1e-4)


def test_gated_delta():
    """The first and the last group of heads beside the same heads alone: the forward and the
    chains are the same kernels on the same values, dq, dk and the gates' gradients may be
    summed in another order."""
    h, groups, dk, dv = 128, 8, 64, 256
    n = (2 ** 31 + 2 ** 27) // (h * dv)
    randn = _randn(2)
    unit = torch.nn.functional.normalize
    wide = randn(1, n, h * dv + 8)
    t = {"q": unit(randn(1, n, groups, dk), dim=-1), "k": unit(randn(1, n, groups, dk), dim=-1),
         "v": wide[..., :h * dv].unflatten(-1, (h, dv)),
         "g": -0.1 * randn(1, n, h, dtype=F32).abs(), "beta": torch.sigmoid(randn(1, n, h, dtype=F32))}
    dy, state, dlast = randn(1, n, h, dv), randn(1, h, dv, dk, dtype=F32), randn(1, h, dv, dk, dtype=F32)

    def both(t, dy, state, dlast):
        five = (1, n, t["v"].shape[2], dk, dv)
        kept = torch.empty(binding.ssm_gated_delta_checkpoint_bytes(*five), dtype=torch.uint8, device="cuda")
        y, last = binding.ssm_gated_delta_fwd(*t.values(), initial_state=state, checkpoints=kept)
        g = binding.ssm_gated_delta_bwd(*t.values(), dy, initial_state=state, dfinal_state=dlast, checkpoints=kept)
        return y, last, g

    y, last, g = both(t, dy, state, dlast)
    for group in (0, groups - 1):
        at = slice(group * h // groups, (group + 1) * h // groups)
        own = {k: (x[:, :, group:group + 1] if k in "qk" else x[:, :, at]).contiguous() for k, x in t.items()}
        y1, last1, g1 = both(own, dy[:, :, at].contiguous(), state[:, at].contiguous(), dlast[:, at].contiguous())
        assert torch.equal(y[:, :, at], y1) and torch.equal(last[:, at], last1)
        assert torch.equal(g["dv"][:, :, at], g1["dv"])
        assert torch.equal(g["dinitial_state"][:, at], g1["dinitial_state"])
        for name in ("dg", "dbeta"):
            near(g[name][:, :, at], to64(g1[name]), 2 * GATES)
        for name in ("dq", "dk"):
            near(g[name][:, :, group:group + 1], to64(g1[name]), 2 * BWD + ROUND)


def test_gated_delta_walked():
    """Decode: states of more than 2^31 elements, updated in place."""
    b, h, d = 2176, 64, 128
    randn = _randn(3)
    unit = torch.nn.functional.normalize
    q, k = unit(randn(b, 1, h, d), dim=-1), unit(randn(b, 1, h, d), dim=-1)
    v, g, beta = randn(b, 1, h, d), -0.1 * randn(b, 1, h, dtype=F32).abs(), torch.sigmoid(randn(b, 1, h, dtype=F32))
    state = randn(b, h, d, d, dtype=F32)
    ends = [0, 2 ** 31 // (h * d * d), b - 1]
    was = [to64(state[i:i + 1]) for i in ends]
    y, _ = binding.ssm_gated_delta_fwd(q, k, v, g, beta, initial_state=state, final_state=state)
    for i, s in zip(ends, was):
        y_ref, s_ref, _ = H.delta_fwd(*(to64(x[i:i + 1]) for x in (q, k, v, g, beta)), s)
        near(y[i:i + 1], y_ref, 2.5e-3)
        near(state[i:i + 1], s_ref, 2e-6)
