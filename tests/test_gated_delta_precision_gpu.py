"""Gated delta rule: what the results are accurate to, beyond sizes and masks."""
import numpy as np
import pytest
import torch

from tests.helpers import to64
from tests.test_gated_delta_gpu import BF16, F32, cuda, forward, inputs, kept_for, reference

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
