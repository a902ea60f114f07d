"""Gated delta rule (ssm_gated_delta_fwd, _bwd) against the plain 64-bit form on the same
inputs, step by step.

Tolerances, derived, as parts of the 2-norm.  Walked sequences are fp32 sums of up to 128
products and as many again for u, 2^-24 a rounding, carried on by a state that keys of
length one do not let grow: 2e-6.  In chunks an operand enters as two fp16, 2^-22 of it off
at most, three in a row (the state, what each step is off it, and their product's left
factor), and the tensor cores' sums of up to 3 x 8 parts are cut, not rounded, 2^-23 each in
one direction: 3 * 2^-22 + 24 * 2^-23 = 3.6e-6 at most, and a third of it on average; the
inverse of the chunk's triangle adds its condition, which is below 3 for such keys: 4e-6.
Products that only gradients in bf16 come from have operands rounded to one fp16, half a
step of 2^-11, up to four in a row: 1e-3 at most for dq, dk.  dg and dbeta are sums of such
terms of either sign, of which up to two thirds cancel: 4e-3.  A bf16 result adds 2^-8 at
most and a third of that on average: 2.5e-3."""
import numpy as np
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests import plain64_heads as H
from tests.helpers import to64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FWD, BWD, GATES, ROUND = 4e-6, 1e-3, 4e-3, 2.5e-3


def off(got, ref):
    got = to64(got)
    assert got.shape == ref.shape and np.isfinite(got).all()
    norm = np.linalg.norm(ref)
    return np.linalg.norm(got - ref) / norm if norm else np.linalg.norm(got)


def inputs(b, n, h, groups, dk, dv, state=True, xt=BF16, gt=F32, seed=0, masked=0.1, restart=0.02):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g)

    unit = torch.nn.functional.normalize
    t = {"q": unit(randn(b, n, groups, dk), dim=-1).to(xt),
         "k": unit(randn(b, n, groups, dk) + 0.3 * randn(1, 1, groups, dk), dim=-1).to(xt),
         "v": randn(b, n, h, dv).to(xt)}
    rate = torch.exp(-5 * torch.rand(h, generator=g))
    gate = -rate * torch.nn.functional.softplus(randn(b, n, h))
    beta = torch.sigmoid(randn(b, n, h))
    gate = gate.masked_fill(torch.rand(b, n, h, generator=g) < restart, float("-inf"))
    beta = beta.masked_fill(torch.rand(b, n, h, generator=g) < masked, 0.0)
    t["g"], t["beta"] = gate.to(gt), beta.to(gt)
    t["state"] = randn(b, h, dv, dk) / dk ** 0.5 if state else None
    t["dy"] = randn(b, n, h, dv).to(xt)
    t["dfinal"] = randn(b, h, dv, dk) if state else None
    return t


FIVE = ("q", "k", "v", "g", "beta")


def cuda(t):
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def reference(t):
    a = {k: None if v is None else to64(v) for k, v in t.items()}
    y, last, _ = H.delta_fwd(*(a[k] for k in FIVE), a["state"])
    return y, last


def reference_grads(t):
    a = {k: None if v is None else to64(v) for k, v in t.items()}
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dinitial_state"),
                    H.delta_bwd(*(a[k] for k in FIVE), a["dy"], a["state"], a["dfinal"])))


def forward(c, **kw):
    return binding.ssm_gated_delta_fwd(*(c[k] for k in FIVE), initial_state=c["state"], **kw)


def kept_for(c):
    b, n, h, dv = c["v"].shape
    size = binding.ssm_gated_delta_checkpoint_bytes(b, n, h, c["q"].shape[3], dv)
    return torch.empty(size, dtype=torch.uint8, device="cuda")


def backward(c, **kw):
    return binding.ssm_gated_delta_bwd(*(c[k] for k in FIVE), c["dy"], initial_state=c["state"],
                                       dfinal_state=c["dfinal"], **kw)


def check_grads(got, ref, gt, grad_dtype, state=True):
    rounding = ROUND if grad_dtype == BF16 else 0
    assert off(got["dv"], ref["dv"]) < FWD + rounding
    for name in ("dq", "dk"):
        assert got[name].dtype == grad_dtype
        assert off(got[name], ref[name]) < BWD + rounding, name
    for name in ("dg", "dbeta"):
        assert got[name].dtype == gt
        assert off(got[name], ref[name]) < GATES + (ROUND if gt == BF16 else 0), name
    if state:
        assert off(got["dinitial_state"], ref["dinitial_state"]) < FWD


# lengths around the 10 steps that are walked and around chunks of 64
@pytest.mark.parametrize("n", [1, 2, 9, 10, 11, 16, 17, 63, 64, 65, 128, 129, 320])
@pytest.mark.parametrize("state", [True, False])
def test_lengths(n, state):
    t = inputs(2, n, 3, 3, 128, 64, state, seed=n)
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    yb, lastb = forward(c)
    assert yb.dtype == BF16 and off(yb, y_ref) < ROUND and off(lastb, last_ref) < FWD
    kept = kept_for(c)
    yk, lastk = forward(c, out_dtype=F32, checkpoints=kept)
    assert off(yk, y_ref) < FWD and off(lastk, last_ref) < FWD
    ref = reference_grads(t)
    for kw in ({"checkpoints": kept}, {}):
        check_grads(backward(c, grad_dtype=F32, **kw), ref, F32, F32, state)


@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 40), (24, 256), (64, 64), (64, 128), (72, 72), (96, 200),
                                   (120, 16), (128, 128), (128, 256)])
@pytest.mark.parametrize("h,groups", [(1, 1), (4, 2), (6, 1)])
def test_sizes_and_shared_heads(dk, dv, h, groups):
    t = inputs(1, 150, h, groups, dk, dv, seed=dk + dv, gt=BF16)
    c = cuda(t)
    y_ref, last_ref = reference(t)
    kept = kept_for(c)
    for kw in ({}, {"checkpoints": kept}):
        y, last = forward(c, out_dtype=F32, **kw)
        assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    check_grads(backward(c, checkpoints=kept), reference_grads(t), BF16, BF16)


@pytest.mark.parametrize("dk,dv", [(8, 8), (32, 24), (40, 256), (128, 128)])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_fp32_is_walked(dk, dv, n):
    t = inputs(2, n, 4, 2, dk, dv, xt=F32, seed=n)
    y, last = forward(cuda(t))
    y_ref, last_ref = reference(t)
    assert y.dtype == F32 and off(y, y_ref) < 2e-6 and off(last, last_ref) < 2e-6
    y, _ = forward(cuda(t), out_dtype=BF16)
    assert y.dtype == BF16 and off(y, y_ref) < ROUND


def test_many_heads_and_long_sequences():
    """More heads than SMs, and few on a long sequence (panels of 32 columns)."""
    for b, n, h, dk, dv in ((40, 70, 8, 64, 64), (1, 3000, 2, 128, 128)):
        t = inputs(b, n, h, h, dk, dv, seed=n, restart=0.002)
        c = cuda(t)
        y_ref, last_ref = reference(t)
        y, last = forward(c, out_dtype=F32)
        assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
        y, last = forward(c)
        assert off(y, y_ref) < ROUND and off(last, last_ref) < FWD
        check_grads(backward(c, grad_dtype=F32), reference_grads(t), F32, F32)


@pytest.mark.parametrize("xt,n", [(F32, 9), (BF16, 9), (BF16, 100)])
def test_masked_steps_are_not_looked_at(xt, n):
    t = inputs(2, n, 2, 2, 64, 64, xt=xt, seed=3)
    t["beta"][:, 2:5] = 0
    t["beta"][1, n // 2:] = 0
    y_ref, last_ref = reference(t)
    gone = (t["beta"] == 0)[..., None]
    t["k"], t["v"] = t["k"].masked_fill(gone, float("nan")), t["v"].masked_fill(gone, float("inf"))
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    if xt == BF16:
        g = backward(c, grad_dtype=F32)
        ref = reference_grads(t)
        check_grads(g, ref, F32, F32)
        assert not g["dk"].cpu()[gone.expand_as(t["k"])].any()
        assert not g["dv"].cpu()[gone.expand_as(t["v"])].any() and not g["dbeta"].cpu()[gone[..., 0]].any()


@pytest.mark.parametrize("n", [7, 100])
def test_all_steps_masked(n):
    """A batch whose steps all learn nothing: the state decays, y answers from it."""
    t = inputs(1, n, 2, 1, 64, 64, seed=4, masked=1.1, restart=0)
    assert not t["beta"].any()
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    g = backward(c, grad_dtype=F32)
    ref = reference_grads(t)
    assert off(g["dq"], ref["dq"]) < BWD and off(g["dg"], ref["dg"]) < GATES
    assert not g["dk"].any() and not g["dv"].any() and not g["dbeta"].any()


@pytest.mark.parametrize("xt,n", [(F32, 6), (BF16, 6), (BF16, 130)])
def test_a_restart_forgets_the_state_whatever_it_was(xt, n):
    t = inputs(2, n, 2, 2, 64, 64, xt=xt, seed=5, restart=0)
    t["g"][:, 0] = float("-inf")
    clean = dict(t, state=None)
    t["state"] = torch.full_like(t["state"], float("nan"))
    y, last = forward(cuda(t), out_dtype=F32)
    y_ref, last_ref = reference(clean)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD


@pytest.mark.parametrize("at", [1, 31, 32, 63, 64, 99])
def test_restarts_anywhere_in_a_chunk(at):
    t = inputs(1, 130, 2, 2, 64, 64, seed=6, restart=0)
    t["g"][:, at] = float("-inf")
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    g = backward(c, grad_dtype=F32)
    check_grads(g, reference_grads(t), F32, F32)
    assert not g["dg"][:, at].any()


def test_strong_and_no_decay_and_growth():
    """Gates of 0 and of -50 beside one another; gates above 0 for a while."""
    t = inputs(1, 200, 3, 3, 64, 64, seed=7, restart=0)
    t["g"][..., 0] = 0
    t["g"][..., 1] = torch.where(torch.rand(1, 200) < 0.1, -50.0, 0.0)
    t["g"][..., 2] = torch.where(torch.arange(200)[None] % 100 < 50, 0.1, -0.2)
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    check_grads(backward(c, grad_dtype=F32), reference_grads(t), F32, F32)


def test_nan_gate_reaches_what_follows():
    t = inputs(1, 100, 2, 2, 64, 64, seed=8, restart=0)
    clean, _ = forward(cuda(t), out_dtype=F32)
    t["g"][0, 70, 1] = float("nan")
    y, last = forward(cuda(t), out_dtype=F32)
    assert torch.equal(y[:, :64], clean[:, :64]) and torch.equal(y[..., 0, :], clean[..., 0, :])
    assert y[0, 70:, 1].isnan().all() and last[0, 1].isnan().all() and not last[0, 0].isnan().any()


@pytest.mark.parametrize("alike", [0.5, 1.0])
def test_keys_alike(alike):
    """Keys near one another, beta near 1: the chunk's triangle is far from 1.  For equal keys
    its inverse has two diagonals, of a norm up to 2; in between the norm stays below 1 /
    (1 - alike) = 2 for 0.5: twice the tolerance."""
    t = inputs(1, 200, 2, 2, 64, 64, seed=9, masked=0)
    one = torch.nn.functional.normalize(torch.randn(1, 1, 2, 64), dim=-1)
    rest = torch.nn.functional.normalize(torch.randn(1, 200, 2, 64), dim=-1)
    t["k"] = torch.nn.functional.normalize(alike ** 0.5 * one + (1 - alike) ** 0.5 * rest, dim=-1).to(BF16)
    t["beta"] = 1 - 0.1 * torch.rand(1, 200, 2)
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < 2 * FWD and off(last, last_ref) < 2 * FWD
    got, ref = backward(c, grad_dtype=F32), reference_grads(t)
    for name, tol in (("dq", BWD), ("dk", BWD), ("dv", FWD), ("dinitial_state", FWD), ("dg", GATES),
                      ("dbeta", GATES)):
        assert off(got[name], ref[name]) < 2 * tol, name


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 40])
def test_values_and_states_of_any_size(scale):
    """Operands have a factor per tile: results scale with v and the state exactly."""
    t = inputs(1, 150, 2, 2, 64, 64, seed=10)
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    g = backward(c, grad_dtype=F32)
    c["v"], c["state"] = c["v"] * scale, c["state"] * scale
    y2, last2 = forward(c, out_dtype=F32)
    # (bounds hold to a power of two: the same factors, the same roundings)
    assert torch.equal(y2, y * scale) and torch.equal(last2, last * scale)
    c["v"], c["state"] = c["v"] / scale, c["state"] / scale
    c["dy"], c["dfinal"] = c["dy"] * scale, c["dfinal"] * scale
    g2 = backward(c, grad_dtype=F32)
    for name in ("dq", "dk", "dv", "dinitial_state"):
        assert torch.equal(g2[name], g[name] * scale), name


def test_one_large_value_among_small_ones():
    """A tile's factor follows its largest value: 2^-25 of that is the least that counts."""
    t = inputs(1, 100, 1, 1, 64, 64, seed=11, masked=0)
    t["v"][0, 40, 0, 3] = 3e4
    y, last = forward(cuda(t), out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    others = [c for c in range(64) if c != 3]
    small = np.max(np.abs(to64(y)[..., others] - y_ref[..., others]))
    assert small < 3e4 * 2.0 ** -19


def test_zero_inputs_and_unseen_keys():
    t = inputs(1, 80, 2, 2, 64, 64, seed=12, state=False)
    c = cuda(t)
    for name in ("q", "k", "v"):
        z = dict(c, **{name: torch.zeros_like(c[name])})
        y, last = forward(z, out_dtype=F32)
        assert torch.isfinite(y).all() and torch.isfinite(last).all()
        if name != "q":
            assert not last.any()
        g = backward(z, grad_dtype=F32)
        assert all(torch.isfinite(v).all() for v in g.values())


def test_ranges_of_a_projection():
    t = inputs(2, 90, 4, 2, 64, 64, seed=13)
    wide = torch.randn(2, 90, 128 + 128 + 256 + 8).to(BF16)
    wide[..., :128], wide[..., 128:256], wide[..., 256:512] = (t[n].flatten(2) for n in "qkv")
    wide = wide.cuda()
    kept = wide.clone()
    c = cuda(t)
    plain = forward(c), backward(c)
    c["q"], c["k"] = (wide[..., 128 * i:128 * i + 128].unflatten(-1, (2, 64)) for i in range(2))
    c["v"] = wide[..., 256:512].unflatten(-1, (4, 64))
    ranges = forward(c), backward(c)
    assert all(torch.equal(a, b) for a, b in zip(plain[0], ranges[0]))
    assert all(torch.equal(plain[1][k], ranges[1][k]) for k in plain[1])
    assert torch.equal(wide, kept)
    for one in (c, ):  # a few tokens of the same projection
        short = {k: v if k in ("state", "dfinal") or v is None else v[:, :5] for k, v in one.items()}
        short["g"], short["beta"] = short["g"].contiguous(), short["beta"].contiguous()
        if short["q"].shape[0] == 2:
            with pytest.raises(ValueError):
                forward(short)  # the batches do not follow one another


def test_the_state_in_place_and_token_by_token():
    """One token at a time, the state updated in place, against the whole sequence."""
    t = inputs(3, 40, 4, 4, 128, 64, seed=14)
    c = cuda(t)
    y_ref, last_ref = reference(t)
    state, ys = c["state"].clone(), []
    for i in range(40):
        one = {k: c[k][:, i:i + 1].contiguous() for k in FIVE}
        y, s = forward(dict(one, state=state), final_state=state, out_dtype=F32)
        assert s is state
        ys.append(y)
    assert off(torch.cat(ys, 1), y_ref) < 2e-6 and off(state, last_ref) < 2e-6
    state = c["state"].clone()  # and in chunks
    forward(dict(c, state=state), final_state=state)
    assert off(state, last_ref) < FWD


def test_no_steps_no_batch_no_final_state():
    t = inputs(2, 0, 3, 3, 64, 64)
    c = cuda(t)
    y, last = forward(c)
    assert y.shape == (2, 0, 3, 64) and torch.equal(last, c["state"])
    y, last = forward(dict(c, state=None))
    assert not last.any()
    g = backward(c)
    assert torch.equal(g["dinitial_state"], c["dfinal"])
    c = cuda(inputs(0, 5, 3, 3, 64, 64))
    assert forward(c)[0].shape == (0, 5, 3, 64)
    c = cuda(inputs(1, 70, 2, 2, 64, 64))
    y, last = forward(c, return_final_state=False)
    assert last is None and torch.equal(y, forward(c)[0])


def test_runs_are_bit_equal_on_another_stream_and_in_graphs():
    long, short = (cuda(inputs(2, n, 4, 2, 128, 128, seed=15)) for n in (200, 3))

    def all_of(stream=None):
        kept = kept_for(long)
        outs = list(forward(long, checkpoints=kept, stream=stream))
        outs += list(backward(long, checkpoints=kept, stream=stream).values())
        outs += list(forward(long, stream=stream)) + list(forward(short, stream=stream))
        return outs

    first = all_of()
    assert all(torch.equal(a, b) for a, b in zip(first, all_of()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = all_of(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]  # with workspaces of their own
    captured = []
    for g in graphs:
        with torch.cuda.graph(g):
            captured.append(all_of())
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for outs in (other, *captured):
        assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, do not disturb one another."""
    a, b = (cuda(inputs(1, 500, 8, 8, 128, 128, seed=s)) for s in (16, 17))
    ref = [forward(a), forward(b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, (c, s) in enumerate(zip((a, b), streams)):
            outs[i].append(forward(c, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for y, last in outs[i]:
            assert torch.equal(y, ref[i][0]) and torch.equal(last, ref[i][1])


def test_guards_and_status():
    """Nothing is written outside the outputs (odd sizes), and no wait ran out."""
    t = inputs(2, 77, 6, 2, 72, 40, seed=18, gt=BF16)
    c = cuda(t)
    shapes = {"y": (c["v"].shape, F32), "final_state": (c["state"].shape, F32),
              "dq": (c["q"].shape, BF16), "dk": (c["k"].shape, BF16), "dv": (c["v"].shape, BF16),
              "dg": (c["g"].shape, BF16), "dbeta": (c["g"].shape, BF16),
              "dinitial_state": (c["state"].shape, F32)}
    bufs, views = {}, {}
    for name, (shape, dt) in shapes.items():
        size = int(np.prod(shape))
        bufs[name] = torch.full((size + 128,), 7.0, dtype=dt, device="cuda")
        views[name] = bufs[name][64:64 + size].view(shape)
    five = 2, 77, 6, 72, 40
    sizes = {"kept": binding.ssm_gated_delta_checkpoint_bytes(*five), "ws": 1024,
             "bws": binding.ssm_gated_delta_bwd_workspace_bytes(*five)}
    own = {k: torch.full((n + 512,), 7, dtype=torch.uint8, device="cuda") for k, n in sizes.items()}
    mid = {k: own[k][256:256 + n] for k, n in sizes.items()}
    forward(c, out_dtype=F32, y=views["y"], final_state=views["final_state"], checkpoints=mid["kept"],
            workspace=mid["ws"])
    backward(c, checkpoints=mid["kept"], workspace=mid["bws"],
             out={k: v for k, v in views.items() if k.startswith("d")})
    assert binding.ssm_last_device_status(mid["ws"]) == 0
    assert binding.ssm_last_device_status(mid["bws"]) == 0
    for name, b in bufs.items():
        assert torch.all(b[:64] == 7) and torch.all(b[-64:] == 7), name
    for name, b in own.items():
        assert torch.all(b[:256] == 7) and torch.all(b[-256:] == 7), name
    y_ref, last_ref = reference(t)
    assert off(views["y"], y_ref) < FWD and off(views["final_state"], last_ref) < FWD


@pytest.mark.parametrize("dv", [64, 128, 200])
def test_columns_that_later_steps_do_not_read(dv):
    """Some columns of headdim have no gradient behind a chunk, or far less than others: what
    the chunk itself gives them counts in full."""
    for far in (0.0, 2.0 ** -14):
        t = inputs(1, 150, 4, 2, 64, dv, seed=dv, restart=0)
        t["dy"][:, 64:, :, dv // 2:] *= far
        t["dfinal"][:, :, dv // 2:] *= far
        check_grads(backward(cuda(t), grad_dtype=F32), reference_grads(t), F32, F32)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_reach_their_own_columns(bad):
    """A v that is not finite spoils its column of headdim from its chunk on, a state's or a
    gradient's its column, a q its own y: nothing else, to the same tolerances."""
    t = inputs(1, 200, 2, 2, 64, 128, seed=19)
    y_ref, last_ref = reference(t)
    ref = reference_grads(t)
    keep = [c for c in range(128) if c not in (5, 77)]

    s = {k: None if v is None else v.clone() for k, v in t.items()}
    s["beta"][0, 70] = t["beta"][0, 70] = 0.5
    y_ref, last_ref = reference(t)
    ref = reference_grads(t)
    s["v"][0, 70, 0, 5] = bad
    s["state"][0, 1, 77, 3] = bad
    s["q"][0, 130, 1, 2] = bad
    s["q"][0, 199, 0] = bad
    y, last = forward(cuda(s), out_dtype=F32)
    rows = [i for i in range(200) if i not in (130, 199)]
    assert off(y[:, rows][..., keep], y_ref[:, rows][..., keep]) < FWD
    assert off(last[:, :, keep], last_ref[:, :, keep]) < FWD
    assert off(y[:, :64, 0], y_ref[:, :64, 0]) < FWD  # the chunk before
    assert not torch.isfinite(y[0, 70:, 0, 5]).any() and not torch.isfinite(last[0, 0, 5]).any()
    assert not torch.isfinite(y[0, 130, 1]).any() and not torch.isfinite(y[0, 199, 0]).any()

    s = {k: None if v is None else v.clone() for k, v in t.items()}
    s["dy"][0, 100, 0, 5] = bad
    s["dfinal"][0, 1, 77, 3] = bad
    g = backward(cuda(s), grad_dtype=F32)
    assert off(g["dv"][..., keep], ref["dv"][..., keep]) < FWD
    assert off(g["dinitial_state"][:, :, keep], ref["dinitial_state"][:, :, keep]) < FWD
    assert off(g["dq"][:, 128:, 0], ref["dq"][:, 128:, 0]) < BWD  # the chunks behind
    assert not torch.isfinite(g["dq"][0, 100, 0]).any()
    assert not torch.isfinite(g["dk"][0, 60, 0]).any()


def test_status_of_many_calls():
    """No wait runs out, in either arrangement of the kernels, and results do not change from call
    to call."""
    for h, n, dk, dv, dt in ((1, 200, 64, 40, F32), (6, 150, 16, 40, F32), (6, 400, 128, 64, BF16),
                             (30, 300, 64, 128, BF16), (200, 130, 64, 64, BF16)):
        c = cuda(inputs(1, n, h, h, dk, dv, seed=h))
        ws = torch.empty(binding.ssm_gated_delta_workspace_bytes(1, n, h, dk, dv), dtype=torch.uint8,
                         device="cuda")
        first = forward(c, out_dtype=dt, workspace=ws)
        for _ in range(20):
            again = forward(c, out_dtype=dt, workspace=ws)
            assert binding.ssm_last_device_status(ws) == 0
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("n", [1, 2, 70])
def test_a_first_gate_without_a_state_has_no_gradient(n):
    t = inputs(2, n, 3, 1, 64, 64, state=False, seed=n, restart=0)
    g = backward(cuda(t), grad_dtype=F32)
    assert not g["dg"][:, 0].any()
    assert off(g["dg"], reference_grads(t)["dg"]) < GATES


@pytest.mark.parametrize("b,n,h,groups,dk,dv", [(1, 1, 21, 1, 128, 128), (1, 70, 9, 1, 64, 64), (2, 200, 24, 3, 128, 72),
                                                (3, 1021, 6, 2, 72, 40), (1, 300, 32, 2, 40, 200)])
def test_few_chunks_and_many_heads_of_a_group(b, n, h, groups, dk, dv):
    """A group's heads are shared by CTAs that add up dq and dk."""
    t = inputs(b, n, h, groups, dk, dv, seed=h + n)
    c = cuda(t)
    g = backward(c, grad_dtype=F32)
    check_grads(g, reference_grads(t), F32, F32)
    for _ in range(3):
        again = backward(c, grad_dtype=F32)
        assert all(torch.equal(g[k], again[k]) for k in g)
