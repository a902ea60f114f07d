"""Gated delta rule: what the results are accurate to, beyond sizes and masks."""
import numpy as np
import pytest
import torch

from tests.helpers import to64
from tests.test_gated_delta_gpu import (BF16, BWD, F32, FWD, GATES, ROUND, backward, check_grads, cuda, forward, inputs,
                                        kept_for, off, reference, reference_grads)

pytestmark = pytest.mark.gpu


# walked; records and chains at once; panels of 32 columns; of 64; with what training keeps
@pytest.mark.parametrize("n,h,dk,dv,keep", [(5, 3, 64, 64, False), (300, 2, 128, 128, False), (130, 40, 64, 64, False),
                                            (70, 200, 128, 72, False), (200, 4, 72, 200, True)])
def test_y_in_bf16_is_rounded_once(n, h, dk, dv, keep):
    """y in bf16 is y in fp32, rounded: nothing before has fewer bits."""
    t = inputs(1, n, h, h, dk, dv, seed=n)
    c = cuda(t)
    kw = {"checkpoints": kept_for(c)} if keep else {}
    fine, _ = forward(c, out_dtype=F32, **kw)
    y, _ = forward(c, out_dtype=BF16, **kw)
    assert torch.equal(y, fine.to(BF16))
    # half a step of bf16, beside the products' own: 2^-20 (three operands of two fp16 and the
    # sums) of up to 192 terms of either sign, in sum below 8 times the largest result
    ref = reference(t)[0]
    assert (np.abs(to64(y) - ref) <= np.abs(ref) * 2.0 ** -8 + np.abs(ref).max() * 2.0 ** -17).all()


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("small", [1e-3, 1e-6, 1e-9, 1e-12, 1e-20, 1e-30])
@pytest.mark.parametrize("n,h,dk,dv", [(150, 4, 64, 64), (200, 2, 128, 128), (70, 6, 72, 136)])
def test_small_betas_beside_others(small, gt, n, h, dk, dv):
    """A step that learns next to nothing has a gradient of beta as large as the others': (L k) . e,
    which is not a difference of anything rounded with beta in it.  Its own steps are held to what
    all are: sums of products of either sign of operands rounded to fp16."""
    t = inputs(1, n, h, h // 2, dk, dv, seed=n, gt=gt)
    at = torch.arange(n) % 8 == 3
    t["beta"][:, at] = (small * (0.5 + torch.rand(1, int(at.sum()), h))).to(gt)
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    kept = kept_for(c)
    forward(c, checkpoints=kept)
    for kw in ({}, {"checkpoints": kept}):
        g, ref = backward(c, grad_dtype=F32, **kw), reference_grads(t)
        check_grads(g, ref, gt, F32)
        rounding = ROUND if gt == BF16 else 0
        assert off(g["dbeta"][:, at], ref["dbeta"][:, at.numpy()]) < GATES + rounding
        assert off(g["dv"][:, at], ref["dv"][:, at.numpy()]) < FWD


def test_betas_from_0_to_1_alone():
    """Every step's beta another power of two, down to 2^-100, in no order."""
    t = inputs(1, 320, 2, 2, 64, 64, seed=21, masked=0)
    t["beta"] = 2.0 ** -torch.randint(0, 101, (1, 320, 2)).float()
    g, ref = backward(cuda(t), grad_dtype=F32), reference_grads(t)
    check_grads(g, ref, F32, F32)
    for lo, hi in ((1.0, 2.0 ** -9), (2.0 ** -10, 2.0 ** -40), (2.0 ** -41, 2.0 ** -100)):
        at = ((t["beta"] <= lo) & (t["beta"] >= hi))[0].numpy()
        assert off(g["dbeta"].cpu()[0][torch.from_numpy(at)], ref["dbeta"][0][at]) < GATES


@pytest.mark.parametrize("top", [1.9, 100.0, -1.0])
def test_betas_above_1_and_below_0(top):
    """Short keys: beta k . k stays below 1 (or above -1), so that no state grows faster than its
    gates let it shrink."""
    t = inputs(1, 150, 4, 2, 64, 72, seed=22)
    t["k"] = (t["k"].float() * abs(top) ** -0.5).to(BF16)
    t["beta"] = t["beta"] * top
    if top < 0:
        t["g"] -= 0.7
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    # (below 0 the triangle's inverse grows: 1 + k . k a step, in whose span the gates halve it)
    wide = 2 if top < 0 else 1
    assert off(y, y_ref) < wide * FWD and off(last, last_ref) < wide * FWD
    got, ref = backward(c, grad_dtype=F32), reference_grads(t)
    for name, tol in (("dq", BWD), ("dk", BWD), ("dv", FWD), ("dinitial_state", FWD), ("dg", GATES),
                      ("dbeta", GATES)):
        assert off(got[name], ref[name]) < wide * tol, name


@pytest.mark.parametrize("scale", [2.0 ** -20, 2.0 ** 12, 2.0 ** 30, 2.0 ** 90])
def test_queries_of_any_size(scale):
    """Keys do not lose bits by large queries: y scales with q, the state is untouched."""
    t = inputs(2, 150, 4, 2, 64, 64, seed=23)
    t["q"] = t["q"] * scale
    y_ref, last_ref = reference(t)
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    t["dy"], t["dfinal"] = t["dy"] / scale, t["dfinal"]
    check_grads(backward(cuda(t), grad_dtype=F32), reference_grads(t), F32, F32)


@pytest.mark.parametrize("n,h,dk,dv", [(150, 4, 64, 64), (200, 2, 128, 72), (130, 160, 64, 64)])
@pytest.mark.parametrize("huge", [1e3, 1e10, 3e38])
def test_queries_of_padding_take_no_bits(huge, n, h, dk, dv):
    """A padded batch whose masked steps hold any finite q (memory that nobody wrote): all other
    steps are as exact as without them, forward and gradient (theirs has dy 0)."""
    t = inputs(1, n, h, h // 2, dk, dv, seed=24)
    pad = torch.zeros(1, n, dtype=torch.bool)
    pad[:, n // 2 + 7:] = True
    pad[:, 20:23] = True
    t["beta"], t["g"] = (t[k].masked_fill(pad[..., None], 0.0) for k in ("beta", "g"))
    t["dy"] = t["dy"].masked_fill(pad[..., None, None], 0.0)
    y_ref, last_ref = reference(t)
    ref = reference_grads(t)
    t["q"] = torch.where(pad[..., None, None], (torch.randn(t["q"].shape) * huge).clamp(-3e38, 3e38).to(BF16), t["q"])
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    valid = (~pad[0]).nonzero()[:, 0]
    assert off(y[:, valid], y_ref[:, valid.numpy()]) < FWD and off(last, last_ref) < FWD
    g = backward(c, grad_dtype=F32)
    check_grads(g, ref, F32, F32)


@pytest.mark.parametrize("learners", [0.0, 2.0 ** -9, 1.0])
def test_masked_steps_that_ask(learners):
    """Steps that learn nothing but read: their q, larger or smaller than the others' (whose is small
    or 0 where they only learn), counts; which they are differs from head to head."""
    t = inputs(1, 200, 4, 2, 64, 64, seed=25, masked=0.4)
    t["beta"][:, 64:128] = 0         # a chunk that learns nothing
    t["q"] = torch.where((t["beta"] > 0).any(-1)[..., None, None], t["q"] * learners, t["q"])
    t["q"][:, 1::3] *= 64
    t["q"][:, 2::7] *= 2.0 ** -9
    t["q"][:, 5] = 0
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    g, ref = backward(c, grad_dtype=F32), reference_grads(t)
    check_grads(g, ref, F32, F32)
    for i in (5, 60, 150):
        assert off(g["dq"][:, i], ref["dq"][:, i]) < 2 * BWD  # (one step, not the mean of many)


@pytest.mark.parametrize("sign", [1, -1])
def test_growth_without_gradients(sign):
    """Chunks that grow by e^12 and hold no gradient: they are 0, not 0 times infinity."""
    t = inputs(1, 256, 2, 2, 64, 64, seed=26, restart=0)
    t["g"][:, 64:128, 0], t["g"][:, 192:256, 0] = 0.19, 0.19
    t["g"][:, 128:192, 0] -= 0.2
    t["dy"][:, 64:, 0], t["dfinal"][:, 0] = 0, 0
    t["beta"][:, 64:, 0] *= sign
    g, ref = backward(cuda(t), grad_dtype=F32), reference_grads(t)
    check_grads(g, ref, F32, F32)
    assert not g["dv"][:, 64:, 0].any() and not g["dq"][:, 64:, 0].any()


@pytest.mark.parametrize("nats", [6, 10, 12])
def test_growth_within_a_chunk(nats):
    """Gates above 0: e^nats in 64 steps, whose operands' rows lie as far apart.  Two fp16 hold
    2^-39 of the bound above a tile's largest value, which is up to 2^14 too large here: rows e^12 =
    2^17 smaller are off by 2^-8 of theirs times what they are multiplied with, which is 2^17
    larger than others' but counts once in 64: 2^-17 at most, in the mean of all rows 2 * FWD."""
    t = inputs(1, 192, 2, 2, 64, 64, seed=27, restart=0)
    t["g"][:, 64:128], t["g"][:, 128:] = nats / 64, -nats / 64
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < 2 * FWD and off(last, last_ref) < 2 * FWD
    got, ref = backward(c, grad_dtype=F32), reference_grads(t)
    for name, tol in (("dq", BWD), ("dk", BWD), ("dv", 2 * FWD), ("dinitial_state", 2 * FWD), ("dg", GATES),
                      ("dbeta", GATES)):
        assert off(got[name], ref[name]) < tol, name


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-12])
def test_queries_of_next_to_nothing(size):
    """dq does not depend on q: it is right where q is 0 or nearly, in steps that learn and in a
    chunk that does not, with gradients of y of any size."""
    t = inputs(1, 200, 4, 2, 64, 64, seed=28)
    t["beta"][:, 64:128] = 0
    t["q"] = t["q"] * size
    t["dy"][:, 128:] *= 1e-6
    ref = reference_grads(t)
    g = backward(cuda(t), grad_dtype=F32)
    for at in (slice(0, 64), slice(64, 128), slice(128, 200)):
        assert off(g["dq"][:, at], ref["dq"][:, at]) < BWD
    for name, tol in (("dk", BWD), ("dv", FWD), ("dbeta", GATES)):
        assert off(g[name], ref[name]) < tol, name
    # what restarts leave of it is sum(dy q^T) alone, some 1e-30 or 1e-12.  Such a q is held under the
    # keys' factor, at most 2^13 / max|k|, in fp16, 2^-24 apart: off by 2^-25 / 2^12 max|k| at most
    # each, so the sum over 200 steps of dy (and what is carried on does not grow) by 200 times that
    least = 200 * 2.0 ** -37 * float(t["k"].abs().max() * t["dy"].abs().max()) * ref["dinitial_state"].size ** 0.5
    diff = np.linalg.norm(to64(g["dinitial_state"]) - ref["dinitial_state"])
    assert diff < FWD * np.linalg.norm(ref["dinitial_state"]) + least


@pytest.mark.parametrize("onehot", [False, True])
@pytest.mark.parametrize("big", [300.0, 3e4, 3e6])
def test_a_large_column_beside_others(big, onehot):
    """Two fp16 hold 2^-39 of the bound that a tile's factor comes from.  Of the next state it is at
    most s + 64 * 2 h (v + 128 * 2 k s), with s, v, h, k the largest |S|, |V|, |H|, |K|: 2^16 s for
    one-hot keys (h, k = 1), where no sum is larger than one term: 2^-23 of the largest a chunk, 2^-22
    for two."""
    t = inputs(1, 128, 2, 2, 128, 128, seed=30, masked=0, restart=0)
    if onehot:
        t["k"] = torch.nn.functional.one_hot(torch.randint(0, 128, (1, 128, 2)), 128).to(BF16)
    t["v"][..., 3], t["state"][:, :, 3] = t["v"][..., 3] * big, t["state"][:, :, 3] * big
    y, last = forward(cuda(t), out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < FWD and off(last, last_ref) < FWD
    most = max(float(t["v"].abs().max()), float(t["state"].abs().max()), np.abs(last_ref).max())
    others = [c for c in range(128) if c != 3]
    assert np.abs(to64(last) - last_ref)[:, :, others].max() < most * 2.0 ** -22
    assert np.abs(to64(y) - y_ref)[..., others].max() < most * 2.0 ** -22


@pytest.mark.parametrize("n,h,groups,dk,dv", [(1000, 4, 4, 128, 128), (320, 6, 2, 64, 64), (150, 4, 2, 72, 200)])
def test_what_the_header_says(n, h, groups, dk, dv):
    """y and the state 1e-6; dq, dk and dbeta up to six operands rounded to one fp16 (N, R, U, z or S0,
    L, W), each 2^-11 / sqrt(12) = 1.4e-4 in the mean: 3.5e-4, and a fifth more where roundings of one
    tile add up in a column; dg a sum of such terms of which up to two thirds cancel."""
    t = inputs(2, n, h, groups, dk, dv, seed=n + 1)
    c = cuda(t)
    y, last = forward(c, out_dtype=F32)
    y_ref, last_ref = reference(t)
    assert off(y, y_ref) < 1e-6 and off(last, last_ref) < 1e-6
    g, ref = backward(c, grad_dtype=F32), reference_grads(t)
    for name, tol in (("dv", 1e-6), ("dinitial_state", 1e-6), ("dq", 4.2e-4), ("dk", 4.2e-4), ("dbeta", 4.2e-4),
                      ("dg", 1.2e-3)):
        assert off(g[name], ref[name]) < tol, name
