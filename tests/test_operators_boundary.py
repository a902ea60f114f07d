"""Refusals of the norm, the recurrence and the cross entropy: every call carries an
argument error that the host-side checks catch before anything is launched, on
fake pointers that are never dereferenced."""
import ctypes

import pytest
import torch

from state_space_model_selective_gb300 import binding

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, WS, TIMEOUT, CUDA, ALIAS = range(10)


@pytest.fixture(scope="module")
def L():
    return binding.lib()


def P(i, off=0):
    return ctypes.c_void_p(0x40000000 * (i + 1) + off)


def norm(L, **kw):
    a = dict(x=P(0), res=P(1), w=P(2), eps=1e-5, y=P(3), sum=P(4), rows=8, dim=64, it=1, rt=1, ot=1)
    a.update(kw)
    return L.ssm_add_rmsnorm_fwd(a["x"], a["res"], a["w"], a["eps"], a["y"], a["sum"], a["rows"],
                                 a["dim"], a["it"], a["rt"], a["ot"], None)


def test_norm(L):
    assert norm(L, x=None) == NULL and norm(L, w=None) == NULL and norm(L, y=None) == NULL
    assert norm(L, rows=-1) == SHAPE and norm(L, dim=0) == SHAPE
    assert norm(L, it=5) == DTYPE and norm(L, rt=-1) == DTYPE and norm(L, ot=2) == DTYPE
    assert norm(L, dim=16385) == UNSUP
    assert norm(L, it=0, rt=1) == UNSUP          # a residual narrower than x
    for name in ("x", "res", "w", "y", "sum"):
        assert norm(L, **{name: P(9, 8)}) == ALIGN
    assert norm(L, y=P(0)) == ALIAS and norm(L, y=P(1)) == ALIAS and norm(L, y=P(4)) == ALIAS
    assert norm(L, sum=P(0)) == ALIAS and norm(L, sum=P(1, 64)) == ALIAS  # not the residual itself
    assert norm(L, y=P(2)) == ALIAS
    assert norm(L, rows=0, x=None, y=None) == OK


def quant(L, **kw):
    a = dict(x=P(0), res=P(1), w=P(2), group=128, q=P(3), sc=P(4), sum=P(5), rows=8, dim=256, it=1,
             rt=1)
    a.update(kw)
    return L.ssm_add_rmsnorm_e4m3_fwd(a["x"], a["res"], a["w"], 1e-5, a["group"], a["q"], a["sc"],
                                      a["sum"], a["rows"], a["dim"], a["it"], a["rt"], None)


def test_norm_e4m3(L):
    assert quant(L, q=None) == NULL and quant(L, sc=None) == NULL
    assert quant(L, group=-1) == SHAPE
    for group in (1, 16, 48, 512):
        assert quant(L, group=group) == UNSUP
    assert quant(L, it=3) == DTYPE and quant(L, dim=20000) == UNSUP
    assert quant(L, sc=P(4, 4)) == ALIGN
    assert quant(L, sc=P(3)) == ALIAS and quant(L, q=P(0)) == ALIAS and quant(L, sc=P(5)) == ALIAS
    assert quant(L, rows=0, x=None) == OK


def norm_bwd(L, **kw):
    a = dict(s=P(0), w=P(1), dy=P(2), ds=P(3), dx=P(4), dr=P(5), dw=P(6), rows=8, dim=64, it=1, rt=0,
             dt=1, ws=P(7), n=1 << 30)
    a.update(kw)
    return L.ssm_add_rmsnorm_bwd(a["s"], a["w"], 1e-5, a["dy"], a["ds"], a["dx"], a["dr"], a["dw"],
                                 a["rows"], a["dim"], a["it"], a["rt"], a["dt"], a["ws"], a["n"],
                                 None)


def test_norm_bwd(L):
    for name in ("s", "w", "dy", "dw"):
        assert norm_bwd(L, **{name: None}) == NULL
    assert norm_bwd(L, dx=None, dr=None) == NULL
    assert norm_bwd(L, ws=None) == WS and norm_bwd(L, n=64) == WS
    assert norm_bwd(L, dt=4) == DTYPE and norm_bwd(L, it=0, rt=1) == UNSUP
    assert norm_bwd(L, rows=-2) == SHAPE
    assert norm_bwd(L, dw=P(6, 4)) == ALIGN
    assert norm_bwd(L, dx=P(0)) == ALIAS and norm_bwd(L, dr=P(3)) == ALIAS
    assert norm_bwd(L, dw=P(4)) == ALIAS and norm_bwd(L, n=1 << 29, ws=P(2)) == ALIAS
    assert binding.ssm_add_rmsnorm_bwd_workspace_bytes(-1, 64) == 0
    assert binding.ssm_add_rmsnorm_bwd_workspace_bytes(8, 16385) == 0


def linrec(L, **kw):
    a = dict(f=P(0), x=P(1), z=P(2), sf=64, sx=64, sz=64, h0=P(3), y=P(4), fin=P(5), ck=P(6), batch=2,
             n=200, dim=64, it=1, ot=1, ws=P(7), nb=1 << 28)
    a.update(kw)
    return L.ssm_linrec_fwd(a["f"], a["x"], a["z"], a["sf"], a["sx"], a["sz"], a["h0"], a["y"],
                            a["fin"], a["ck"], a["batch"], a["n"], a["dim"], a["it"], a["ot"],
                            a["ws"], a["nb"], None)


def test_linrec(L):
    for name in ("f", "x", "y"):
        assert linrec(L, **{name: None}) == NULL
    for name in ("batch", "n", "dim"):
        assert linrec(L, **{name: -1}) == SHAPE
    assert linrec(L, sf=63) == SHAPE and linrec(L, sz=1) == SHAPE
    assert linrec(L, it=2) == DTYPE and linrec(L, ot=9) == DTYPE
    assert linrec(L, ws=None) == WS and linrec(L, nb=64) == WS
    assert linrec(L, f=P(0, 1)) == ALIGN             # not even an element's alignment
    assert linrec(L, it=0, x=P(1, 2)) == ALIGN
    assert linrec(L, y=P(4, 8)) == ALIGN and linrec(L, h0=P(3, 4)) == ALIGN
    assert linrec(L, y=P(0)) == ALIAS and linrec(L, fin=P(4)) == ALIAS
    assert linrec(L, fin=P(3, 16)) == ALIAS          # part of the initial state
    assert linrec(L, ck=P(1)) == ALIAS and linrec(L, ws=P(2)) == ALIAS
    assert linrec(L, batch=40000, n=2 ** 31 - 1, dim=64, nb=0) == UNSUP
    assert linrec(L, batch=0, f=None, ws=None) == OK and linrec(L, dim=0, sf=0, ws=None) == OK
    # slices of one projection overlap nothing of their own rows but interleave: inputs may
    assert linrec(L, sf=192, sx=192, sz=192, x=P(0, 128), z=P(0, 256), y=P(0, 128)) == ALIAS
    assert binding.ssm_linrec_workspace_bytes(-1, 5, 5) == 0
    assert binding.ssm_linrec_workspace_bytes(2, 200, 64) >= 256
    assert binding.ssm_linrec_checkpoint_bytes(2, 65, 10) == 2 * 2 * 10 * 4


def linrec_bwd(L, **kw):
    a = dict(f=P(0), x=P(1), z=P(2), sf=64, sx=64, sz=64, h0=P(3), dy=P(4), dfin=P(5), ck=P(6),
             df=P(7), dx=P(8), dz=P(9), dh=P(10), batch=2, n=200, dim=64, it=1, gt=1, ws=P(11),
             nb=1 << 28)
    a.update(kw)
    return L.ssm_linrec_bwd(a["f"], a["x"], a["z"], a["sf"], a["sx"], a["sz"], a["h0"], a["dy"],
                            a["dfin"], a["ck"], a["df"], a["dx"], a["dz"], a["dh"], a["batch"],
                            a["n"], a["dim"], a["it"], a["gt"], a["ws"], a["nb"], None)


def test_linrec_bwd(L):
    for name in ("f", "x", "dy", "df", "dx", "dz"):
        assert linrec_bwd(L, **{name: None}) == NULL
    assert linrec_bwd(L, n=-1) == SHAPE and linrec_bwd(L, sx=10) == SHAPE
    assert linrec_bwd(L, it=7) == DTYPE and linrec_bwd(L, gt=7) == DTYPE
    assert linrec_bwd(L, ws=None) == WS and linrec_bwd(L, nb=1000) == WS
    assert linrec_bwd(L, dy=P(4, 2)) == ALIGN
    assert linrec_bwd(L, df=P(8)) == ALIAS and linrec_bwd(L, dx=P(4)) == ALIAS
    assert linrec_bwd(L, dh=P(3)) == ALIAS and linrec_bwd(L, dz=P(6)) == ALIAS


def ce(L, **kw):
    a = dict(h=P(0), W=P(1), t=P(2), loss=P(3), lse=P(4), tokens=8, dim=64, vocab=100, it=1, ws=P(5),
             n=1 << 28)
    a.update(kw)
    return L.ssm_vocab_ce_fwd(a["h"], a["W"], a["t"], a["loss"], a["lse"], a["tokens"], a["dim"],
                              a["vocab"], a["it"], a["ws"], a["n"], None)


def test_vocab_ce(L):
    for name in ("h", "W", "t", "loss", "lse"):
        assert ce(L, **{name: None}) == NULL
        assert ce(L, **{name: P(9, 8)}) == ALIGN
    assert ce(L, tokens=-1) == SHAPE and ce(L, dim=0) == SHAPE and ce(L, vocab=0) == SHAPE
    assert ce(L, dim=60) == UNSUP and ce(L, it=0) == UNSUP and ce(L, it=4) == DTYPE
    assert ce(L, ws=None) == WS and ce(L, n=10) == WS
    assert ce(L, loss=P(4)) == ALIAS and ce(L, lse=P(0)) == ALIAS and ce(L, ws=P(1)) == ALIAS
    assert ce(L, tokens=0, h=None) == OK
    assert binding.ssm_vocab_ce_workspace_bytes(8, 60, 100) == 0


def ce_bwd(L, **kw):
    a = dict(h=P(0), W=P(1), t=P(2), lse=P(3), dl=P(4), dh=P(5), dW=P(6), tokens=8, dim=64, vocab=100,
             it=1, gt=1, ws=P(7), n=1 << 28)
    a.update(kw)
    return L.ssm_vocab_ce_bwd(a["h"], a["W"], a["t"], a["lse"], a["dl"], a["dh"], a["dW"],
                              a["tokens"], a["dim"], a["vocab"], a["it"], a["gt"], a["ws"], a["n"],
                              None)


def test_vocab_ce_bwd(L):
    for name in ("h", "W", "t", "lse", "dl", "dh", "dW"):
        assert ce_bwd(L, **{name: None}) == NULL
        assert ce_bwd(L, **{name: P(9, 8)}) == ALIGN
    assert ce_bwd(L, tokens=-1) == SHAPE and ce_bwd(L, vocab=-5) == SHAPE
    assert ce_bwd(L, dim=12) == UNSUP and ce_bwd(L, it=0) == UNSUP and ce_bwd(L, gt=3) == DTYPE
    assert ce_bwd(L, ws=None) == WS and ce_bwd(L, n=256) == WS
    assert ce_bwd(L, dh=P(0)) == ALIAS and ce_bwd(L, dW=P(1)) == ALIAS and ce_bwd(L, dW=P(5)) == ALIAS
    # a piece of the vocabulary, not all of it, once all would pass 256 MB
    whole = 65536 * 50257 * 2
    assert binding.ssm_vocab_ce_bwd_workspace_bytes(65536, 2048, 50257) < whole // 3


def test_binding_takes_cuda_tensors_only():
    t = torch.zeros(2, 3, 8)
    w = torch.ones(8)
    for call in (lambda: binding.ssm_add_rmsnorm_fwd(t, w),
                 lambda: binding.ssm_add_rmsnorm_e4m3_fwd(t, w),
                 lambda: binding.ssm_add_rmsnorm_bwd(t, t, w),
                 lambda: binding.ssm_linrec_fwd(t, t),
                 lambda: binding.ssm_linrec_bwd(t, t, t),
                 lambda: binding.ssm_vocab_ce_fwd(t[0], t[1], torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(TypeError):
            call()


def test_step_strides_of_slices():
    """The recurrence's inputs: contiguous, or a range of the last dimension of a
    contiguous tensor; anything else is refused (pure stride logic)."""
    class Cuda(torch.Tensor):
        is_cuda = True

    def steps(t):
        return binding._steps(t.as_subclass(Cuda), "f", t.dtype, t.shape)

    big = torch.zeros(3, 5, 48)
    assert steps(big) == 48 and steps(big[..., 16:32]) == 48
    assert steps(big[:1, :, :16]) == 48 and steps(big[:, :1, :16]) == 240
    assert steps(big[:1, :1, :7]) == 7 and steps(big[:, :, :1]) == 48
    for bad in (big.transpose(0, 1), big[:, :, ::2], big[:, ::2], big[:, 1:], big[:, :, :1].expand(3, 5, 9)):
        with pytest.raises(ValueError):
            steps(bad)


def test_vocab_ce_sizes_near_two_to_the_31(L):
    """All three sizes are counted in ints: what would pass them once rounded up to tiles
    or pieces is refused, before the workspace is looked at."""
    most = 2 ** 31 - 1
    for sizes in ({"tokens": most, "vocab": 1}, {"tokens": most - 255, "vocab": 1},
                  {"tokens": 1, "vocab": most}, {"tokens": 2 ** 30 + 1, "vocab": 1},
                  {"tokens": 1, "vocab": 1, "dim": 2 ** 31 - 8}):
        sizes = {"dim": 8, **sizes}
        assert ce(L, n=0, **sizes) == UNSUP and ce_bwd(L, n=0, **sizes) == UNSUP
        three = sizes["tokens"], sizes["dim"], sizes["vocab"]
        assert binding.ssm_vocab_ce_workspace_bytes(*three) == 0
        assert binding.ssm_vocab_ce_bwd_workspace_bytes(*three) == 0
    assert ce(L, tokens=2 ** 30, vocab=1, dim=8, n=0) == WS
    assert ce(L, tokens=1, vocab=2 ** 30, dim=8, n=0) == WS


def test_linrec_sizes_near_two_to_the_31(L):
    """The steps to the end of a sequence's last tile are counted in an int: sequences whose
    last tile would pass it are refused, before the workspace is looked at."""
    for n in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 128):
        sizes = {"batch": 1, "n": n, "dim": 1, "sf": 1, "sx": 1, "sz": 1, "nb": 0}
        assert linrec(L, **sizes) == UNSUP and linrec_bwd(L, **sizes) == UNSUP
        assert binding.ssm_linrec_workspace_bytes(1, n, 1) == 0
        assert binding.ssm_linrec_bwd_workspace_bytes(1, n, 1) == 0
    assert linrec(L, batch=1, n=2 ** 31 - 129, dim=1, nb=0) == WS
    wide = 2 ** 31 - 1
    assert linrec(L, batch=0, n=1, dim=wide, sf=wide, sx=wide, sz=wide, nb=0) == UNSUP
