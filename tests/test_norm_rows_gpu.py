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


@pytest.mark.parametrize("dim", [7, 100, 257, 1097, 5001])
@pytest.mark.parametrize("xt,rt", [(F32, F32), (BF16, F32), (BF16, BF16)],
                         ids=["f32", "bf16-f32", "bf16"])
def test_sum_in_the_residuals_place_at_odd_widths(dim, xt, rt):
    """Rows share 16-byte units with their neighbours, which other CTAs replace meanwhile."""
    rows = 2 * _fwd_rows(dim) + 3
    x, res, w, _, _ = (t.cuda() for t in _inputs(rows, dim, xt, rt, dim + 2))
    y, s = binding.ssm_add_rmsnorm_fwd(x, w, res, eps=EPS)
    q, scales, _ = binding.ssm_add_rmsnorm_e4m3_fwd(x, w, res, eps=EPS, group=32)
    for _ in range(3):
        stream = res.clone()
        y2, _ = binding.ssm_add_rmsnorm_fwd(x, w, stream, eps=EPS, sum_out=stream)
        assert torch.equal(y2, y) and torch.equal(stream, s)
        stream = res.clone()
        q2, scales2, _ = binding.ssm_add_rmsnorm_e4m3_fwd(x, w, stream, eps=EPS, group=32,
                                                          sum_out=stream)
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))
        assert torch.equal(scales2, scales) and torch.equal(stream, s)


@pytest.mark.parametrize("dim", [7, 100, 257, 1097, 5001])
@pytest.mark.parametrize("xt", [F32, BF16], ids=["f32", "bf16"])
def test_rows_of_nan_and_infinities_between_others(dim, xt):
    """Every third row is NaN, every fifth infinite in one place: the rows beside them, which
    share units with them, are what they are without."""
    rows = 45
    x, res, w, dy, ds = _inputs(rows, dim, xt, xt, dim + 3)
    dy = dy.to(xt)
    bad = torch.zeros(rows, dtype=torch.bool)
    bad[::3], bad[1::5] = True, True
    x2, dy2 = x.clone(), dy.clone()
    x2[::3], dy2[::3] = float("nan"), float("nan")
    x2[1::5, dim - 1], x2[1::5, 0] = float("inf"), float("-inf")

    def all_of(x, dy):
        y, s = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
        q, sc, _ = binding.ssm_add_rmsnorm_e4m3_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS, group=32)
        g = binding.ssm_add_rmsnorm_bwd(dy.cuda(), s, w.cuda(), dsum=ds.cuda(), eps=EPS)
        return y, s, q.float(), sc, g["dx"]

    for a, b in zip(all_of(x2, dy2), all_of(x, dy)):
        a, b = a.cpu(), b.cpu()
        assert torch.equal(a[~bad], b[~bad]) and not a[bad].isfinite().all()
