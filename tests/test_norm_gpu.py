"""RMS norm with the residual's addition (ssm_add_rmsnorm_fwd, _e4m3_fwd, _bwd)
against the plain 64-bit form on the same inputs.

Tolerances, derived: fp32 outputs carry a sum of `dim` squares (relative error
at most about log2(dim) roundings after the tree) and about six roundings a
value, so 4e-6 of the row's largest value; dweight adds a sum over rows,
1e-5 of its largest value.  A bf16 output adds half an ulp, 2^-8 of the value.
An e4m3 value may differ from the correctly rounded one only where y * 448 /
amax lies within 1e-5 of a rounding boundary, and then by one step of the grid."""
import numpy as np
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests import plain64 as P
from tests.helpers import to64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def _near(got, ref, dtype, what, tol=4e-6):
    got = to64(got)
    assert np.all(np.isfinite(got)), what
    scale = np.max(np.abs(ref), axis=-1, keepdims=True)
    lim = tol * scale + (2.0 ** -8 * np.abs(ref) * (1 + 1e-3) if dtype == BF16 else 0.0)
    bad = np.abs(got - ref) > lim
    assert not bad.any(), (what, float(np.max(np.abs(got - ref) - lim)), int(bad.sum()))


def _inputs(rows, dim, xt, rt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, dim, generator=g).to(xt)
    res = (3 * torch.randn(rows, dim, generator=g)).to(rt)
    w = 1 + 0.2 * torch.randn(dim, generator=g)
    dy, ds = torch.randn(rows, dim, generator=g), torch.randn(rows, dim, generator=g).to(rt)
    return x, res, w, dy, ds


# one element; one short of, at and past a warp's block of 256; widths with and
# without 16-byte rows; several warps; past 32 blocks (two blocks a warp); the limit
DIMS = [1, 7, 31, 64, 255, 256, 257, 264, 513, 1537, 2048, 5120, 8200, 8201, 16384]
TYPES = [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, BF16), (BF16, F32, F32),
         (F32, F32, BF16), (BF16, BF16, F32)]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(v)[6:] for v in t))
def test_forward_and_gradient(dim, types):
    xt, rt, yt = types
    rows = 5 if dim > 300 else 37
    x, res, w, dy, ds = _inputs(rows, dim, xt, rt, dim)
    y, s = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS, out_dtype=yt)
    y_ref, s_ref = P.norm_fwd(to64(x), to64(res), to64(w), EPS)
    assert y.dtype == yt and s.dtype == rt
    _near(y, y_ref, yt, "y")
    _near(s, s_ref, rt, "sum", 1e-6)
    dy = dy.to(yt)
    g = binding.ssm_add_rmsnorm_bwd(dy.cuda(), s, w.cuda(), dsum=ds.cuda(), eps=EPS, x_dtype=xt)
    dx_ref, dw_ref = P.norm_bwd(to64(s), to64(w), EPS, to64(dy), to64(ds))
    _near(g["dx"], dx_ref, xt, "dx")
    _near(g["dresidual"], dx_ref, rt, "dresidual")
    assert g["dx"].dtype == xt and g["dresidual"].dtype == rt
    _near(g["dweight"], dw_ref, F32, "dweight", 1e-5)


@pytest.mark.parametrize("rows", [0, 1, 3, 4, 5, 609, 1300])
def test_row_counts(rows):
    """Several rows to a CTA with an incomplete last one; more rows than the
    gradient's CTAs; none at all (dweight is 0)."""
    for dim in (96, 520):
        x, res, w, dy, ds = _inputs(rows, dim, F32, F32, rows)
        y, s = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
        g = binding.ssm_add_rmsnorm_bwd(dy.cuda(), s, w.cuda(), eps=EPS)
        if rows == 0:
            assert y.shape == (0, dim) and not g["dweight"].any()
            continue
        y_ref, s_ref = P.norm_fwd(to64(x), to64(res), to64(w), EPS)
        dx_ref, dw_ref = P.norm_bwd(s_ref, to64(w), EPS, to64(dy))
        _near(y, y_ref, F32, "y")
        _near(g["dx"], dx_ref, F32, "dx")
        _near(g["dweight"], dw_ref, F32, "dweight", 1e-5)


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [5, 32, 256, 300, 1000, 1537, 8704, 9001])
@pytest.mark.parametrize("xt", [F32, BF16], ids=["f32", "bf16"])
def test_e4m3(dim, group, xt):
    rows = 6
    x, res, w, _, _ = _inputs(rows, dim, xt, xt, dim + group)
    x[2], res[2] = 0, 0                       # a row of zeros
    if dim > 40:
        x[3, :40], res[3, :40] = 0, 0         # a whole group of zeros
    q, scales, s = binding.ssm_add_rmsnorm_e4m3_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS,
                                                    group=group)
    y_ref, s_ref = P.norm_fwd(to64(x), to64(res), to64(w), EPS)
    _near(s, s_ref, xt, "sum", 1e-6)
    amax = P.group_amax(y_ref, group)
    np.testing.assert_allclose(to64(scales), amax / 448.0, rtol=4e-6)
    full = np.repeat(amax, group or dim, 1)[:, :dim]
    v = np.divide(y_ref * 448.0, full, out=np.zeros_like(y_ref), where=full > 0)
    got = to64(q.float())
    lo, hi = P.e4m3_round(v * (1 - 1e-5)), P.e4m3_round(v * (1 + 1e-5))
    assert np.all((got == P.e4m3_round(v)) | (got == lo) | (got == hi))
    assert not got[2].any() and not to64(scales)[2].any()


def test_no_residual_and_no_sum():
    x, _, w, dy, _ = _inputs(9, 640, BF16, BF16, 3)
    y, s = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), eps=EPS, return_sum=False)
    assert s is None
    _near(y, P.norm_fwd(to64(x), None, to64(w), EPS)[0], BF16, "y")
    # the sum in 32 bits without a residual: the start of a 32-bit residual stream
    y2, s2 = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), eps=EPS, sum_dtype=F32)
    assert s2.dtype == F32 and torch.equal(s2.cpu(), x.float()) and torch.equal(y, y2)


def test_sum_replaces_the_residual():
    x, res, w, _, _ = _inputs(33, 1096, BF16, F32, 4)
    y, s = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    stream = res.cuda()
    y2, s2 = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), stream, eps=EPS, sum_out=stream)
    assert s2 is stream and torch.equal(stream, s) and torch.equal(y, y2)


def test_leading_dimensions_and_zero_rows_of_values():
    """(batch, seqlen, dim) inputs; a row of zeros gives zeros (eps holds the
    quotient), its gradient dy w / sqrt(eps)."""
    x, res, w, dy, _ = _inputs(12, 264, F32, F32, 5)
    x[7], res[7] = 0, 0
    y, s = binding.ssm_add_rmsnorm_fwd(x.view(3, 4, 264).cuda(), w.cuda(),
                                       res.view(3, 4, 264).cuda(), eps=EPS)
    assert y.shape == (3, 4, 264) and not y[1, 3].any()
    g = binding.ssm_add_rmsnorm_bwd(dy.view(3, 4, 264).cuda(), s, w.cuda(), eps=EPS)
    dx_ref, dw_ref = P.norm_bwd(to64(x + res), to64(w), EPS, to64(dy))
    _near(g["dx"].view(12, 264), dx_ref, F32, "dx")
    _near(g["dweight"], dw_ref, F32, "dweight", 1e-5)


def test_nan_and_infinity_stay_in_their_row():
    x, res, w, _, _ = _inputs(4, 512, F32, F32, 6)
    x[1, 100], x[2, 5] = float("nan"), float("inf")
    y, _ = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    q, scales, _ = binding.ssm_add_rmsnorm_e4m3_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    y_ref, _ = P.norm_fwd(to64(x)[[0, 3]], to64(res)[[0, 3]], to64(w), EPS)
    _near(y[[0, 3]], y_ref, F32, "y")
    assert y[1].isnan().all() and y[2, 5].isnan()
    assert scales[[0, 3]].isfinite().all() and scales[1].isnan().all()
    assert q.float()[1].isnan().all() and q.float()[[0, 3]].isfinite().all()


def test_runs_are_bit_equal_and_on_another_stream():
    x, res, w, dy, _ = (t.cuda() for t in _inputs(2000, 1056, BF16, BF16, 7))
    dy = dy.to(BF16)
    torch.cuda.synchronize()
    first = binding.ssm_add_rmsnorm_bwd(dy, x, w, eps=EPS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [binding.ssm_add_rmsnorm_bwd(dy, x, w, eps=EPS, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    for g in again:
        assert torch.equal(g["dx"], first["dx"]) and torch.equal(g["dweight"], first["dweight"])


@pytest.mark.parametrize("dim", [7, 64, 96, 128, 200, 520])
@pytest.mark.parametrize("rows", [1, 3, 5, 33])
def test_gradient_without_eps(dim, rows):
    """eps = 0: rows of values are well defined, and what a warp holds in the place of rows
    past the last one does not reach dweight."""
    x, res, w, dy, ds = _inputs(rows, dim, F32, F32, rows + dim)
    y, s = binding.ssm_add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=0.0)
    _near(y, P.norm_fwd(to64(x), to64(res), to64(w), 0.0)[0], F32, "y")
    g = binding.ssm_add_rmsnorm_bwd(dy.cuda(), s, w.cuda(), dsum=ds.cuda(), eps=0.0)
    dx_ref, dw_ref = P.norm_bwd(to64(s), to64(w), 0.0, to64(dy), to64(ds))
    _near(g["dx"], dx_ref, F32, "dx")
    _near(g["dweight"], dw_ref, F32, "dweight", 1e-5)


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("dim", [40, 300, 512, 9001])
@pytest.mark.parametrize("exponent", [127, 126, 119, 60, -60, -119, -121, -125, -140])
def test_e4m3_of_extreme_groups(dim, group, exponent):
    """Groups whose largest magnitude is near either end of fp32's range are scaled like any:
    q = e4m3(y * (448 / amax)) for every amax.  y itself is rounded to a multiple of 2^-149
    down there, which q may show, and so may the scale."""
    g = torch.Generator().manual_seed(dim + group)
    x = torch.where(torch.rand(5, dim, generator=g) < 0.5, -1.0, 1.0)  # y = x * w
    w = ((2 * torch.rand(dim, generator=g).double() - 1) * 1.9 * 2.0 ** exponent).float()
    q, scales, _ = binding.ssm_add_rmsnorm_e4m3_fwd(x.cuda(), w.cuda(), eps=0.0, group=group)
    y_ref, _ = P.norm_fwd(to64(x), None, to64(w), 0.0)
    amax = P.group_amax(y_ref, group)
    np.testing.assert_allclose(to64(scales), amax / 448.0, rtol=4e-6, atol=2.0 ** -148)
    full = np.repeat(amax, group or dim, 1)[:, :dim]
    v = y_ref * (448.0 / full)
    off = 1e-5 * np.abs(v) + 2 * 448.0 * 2.0 ** -149 / full
    got = to64(q.float())
    assert np.all((got >= P.e4m3_round(v - off)) & (got <= P.e4m3_round(v + off)))
