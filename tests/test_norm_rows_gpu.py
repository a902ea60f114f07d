"""The norm's kernels past their first row: resident CTAs (with one warp or less to a row,
their warps) walk the rows, with the next row's loads in flight, two buffers for their
sums, the groups' maxima cleared from row to row, and the weight's gradient kept over them.
Every case here gives each CTA three rows or more; tolerances as in test_norm_gpu."""
import numpy as np
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests import plain64 as P
from tests.helpers import to64
from tests.test_norm_gpu import BF16, EPS, F32, _inputs, _near

pytestmark = pytest.mark.gpu

SMS = 152


def _chunks(dim):
    """Pieces of 8 elements a row may touch."""
    return -(-dim // 8) + (1 if dim % 8 else 0)


def _at_once(dim, most_threads, per_lane):
    """Rows that are in work at once, from how the kernels are laid out: 8, 16 or 32 lanes to a
    row of up to 32 pieces, eight such warps to a CTA, else a CTA of whole warps."""
    n = _chunks(dim)
    if n <= 32:
        lanes = 8 if n <= 8 else 16 if n <= 16 else 32
        return SMS * (most_threads // 256) * 8 * (32 // lanes)
    return SMS * max(1, most_threads // (32 * -(-n // (32 * per_lane))))


def _fwd_rows(dim):
    return _at_once(dim, 1024, 1 if _chunks(dim) <= (544 if dim % 8 else 1024) else 4)


def _bwd_rows(dim):
    n = _chunks(dim)
    return _at_once(dim, 640, 1 if n <= 512 else 2 if n <= 1024 else 4)


# less than a warp, a warp, several; one, two and four pieces to a lane; each with and
# without 16-byte rows
DIMS = [7, 64, 96, 100, 200, 255, 256, 520, 1537, 2048, 4104, 5120, 5121, 8201, 16384]
TYPES = [(F32, F32), (BF16, F32), (BF16, BF16)]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16-f32", "bf16"])
def test_forward_walks(dim, types):
    xt, rt = types
    rows = 3 * _fwd_rows(dim) + 5
    x, res, w, _, _ = _inputs(rows, dim, xt, rt, dim)
    y, s = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    y_ref, s_ref = P.norm_fwd(to64(x), to64(res), to64(w), EPS)
    _near(y, y_ref, xt, "y")
    _near(s, s_ref, rt, "sum", 1e-6)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("types", TYPES, ids=["f32", "bf16-f32", "bf16"])
def test_gradient_walks(dim, types):
    xt, rt = types
    rows = 3 * _bwd_rows(dim) + 5
    _, s, w, dy, ds = _inputs(rows, dim, xt, rt, dim + 1)
    dy = dy.to(xt)
    for dsum in (ds, None):
        g = binding.ssm_add_rmsnorm_bwd(dy.cuda(), s.cuda(), w.cuda(), eps=EPS, x_dtype=xt,
                                        dsum=None if dsum is None else dsum.cuda())
        dx_ref, dw_ref = P.norm_bwd(to64(s), to64(w), EPS, to64(dy),
                                    None if dsum is None else to64(dsum))
        _near(g["dx"], dx_ref, xt, "dx")
        _near(g["dresidual"], dx_ref, rt, "dresidual")
        _near(g["dweight"], dw_ref, F32, "dweight", 1e-5)


@pytest.mark.parametrize("group", [0, 32, 256])
@pytest.mark.parametrize("dim", [7, 96, 300, 1000, 1537, 2048, 9001])
@pytest.mark.parametrize("xt", [F32, BF16], ids=["f32", "bf16"])
def test_e4m3_walks(dim, group, xt):
    """Rows of very different sizes after one another: a maximum left from the row before
    would show."""
    rows = 3 * _fwd_rows(dim) + 5
    x, _, w, _, _ = _inputs(rows, dim, xt, xt, dim + group)
    size = 4.0 ** -(torch.arange(rows) // _fwd_rows(dim))  # each turn's rows are smaller
    x = (x.float() * size[:, None]).to(xt)
    eps = 1.0  # so that y's size follows the row's
    q, scales, _ = binding.ssm_add_rmsnorm_e4m3_fwd(x.cuda(), w.cuda(), eps=eps, group=group)
    y_ref, _ = P.norm_fwd(to64(x), None, to64(w), eps)
    amax = P.group_amax(y_ref, group)
    np.testing.assert_allclose(to64(scales), amax / 448.0, rtol=4e-6)
    full = np.repeat(amax, group or dim, 1)[:, :dim]
    v = y_ref * 448.0 / full
    got = to64(q.float())
    assert np.all((got == P.e4m3_round(v)) | (got == P.e4m3_round(v * (1 - 1e-5))) |
                  (got == P.e4m3_round(v * (1 + 1e-5))))
