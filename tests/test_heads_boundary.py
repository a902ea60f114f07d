"""Refusals of the norms of heads and of the gated delta rule: every call carries an argument
error that the host-side checks catch before anything is launched, on fake pointers that are
never dereferenced."""
import ctypes

import pytest
import torch

from state_space_model_selective_gb300 import binding

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, WS, TIMEOUT, CUDA, ALIAS = range(10)
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    return binding.lib()


def P(i, off=0):
    return ctypes.c_void_p(0x40000000 * (i + 1) + off)


def qk(L, **kw):
    a = dict(q=P(0), k=P(1), qs=128, ks=64, qw=P(2), kw=P(3), pos=P(4), freq=P(5), eps=1e-5, rot=64,
             inter=0, qo=P(6), ko=P(7), tokens=8, hq=2, hk=1, dim=64, it=1, ot=1)
    a.update(kw)
    return L.ssm_qk_norm_rope_fwd(*a.values(), None)


def test_qk(L):
    for name in ("q", "k", "pos", "freq", "qo", "ko"):
        assert qk(L, **{name: None}) == NULL, name
    assert qk(L, tokens=-1) == SHAPE and qk(L, hq=-1) == SHAPE and qk(L, hk=-1) == SHAPE
    assert qk(L, dim=0) == SHAPE and qk(L, rot=-2) == SHAPE and qk(L, rot=66) == SHAPE
    assert qk(L, rot=63) == SHAPE and qk(L, inter=2) == SHAPE
    assert qk(L, qs=127) == SHAPE and qk(L, ks=63) == SHAPE
    assert qk(L, it=2) == DTYPE and qk(L, ot=-1) == DTYPE
    assert qk(L, dim=60, rot=60) == UNSUP and qk(L, dim=264, rot=0, qs=528, ks=264) == UNSUP
    assert qk(L, hq=5000, qs=1 << 20) == UNSUP
    assert qk(L, q=P(0, 1)) == ALIGN and qk(L, k=P(1, 3)) == ALIGN  # (elements may lie anywhere)
    for name in ("qw", "kw", "freq", "qo", "ko"):
        assert qk(L, **{name: P(9, 8)}) == ALIGN, name
    assert qk(L, pos=P(9, 4)) == ALIGN
    for name in ("q", "k", "qw", "kw", "pos", "freq"):
        at = {"q": 0, "k": 1, "qw": 2, "kw": 3, "pos": 4, "freq": 5}[name]
        assert qk(L, qo=P(at)) == ALIAS and qk(L, ko=P(at)) == ALIAS, name
    assert qk(L, qo=P(7, 64)) == ALIAS
    # a range of a wide projection: the last token's heads end inside it
    assert qk(L, qs=4096, qo=P(0, 7 * 4096 * 2 + 240)) == ALIAS
    assert qk(L, tokens=0, q=None, k=None) == OK and qk(L, hq=0, hk=0, q=None) == OK


def qk_bwd(L, **kw):
    a = dict(dqo=P(0), dko=P(1), q=P(2), k=P(3), qs=128, ks=64, qw=P(4), kw=P(5), pos=P(6),
             freq=P(7), eps=1e-5, rot=64, inter=0, dq=P(8), dk=P(9), dqw=P(10), dkw=P(11), tokens=8,
             hq=2, hk=1, dim=64, it=1, ot=1, ws=P(12), n=1 << 28)
    a.update(kw)
    return L.ssm_qk_norm_rope_bwd(*a.values(), None)


def test_qk_bwd(L):
    for name in ("dqo", "dko", "q", "k", "pos", "freq", "dq", "dk"):
        assert qk_bwd(L, **{name: None}) == NULL, name
    need = binding.ssm_qk_norm_rope_bwd_workspace_bytes(8, 2, 1, 64)
    assert need > 0 and qk_bwd(L, ws=None) == WS and qk_bwd(L, n=need - 1) == WS
    assert qk_bwd(L, ws=P(12, 8)) == ALIGN
    for name in ("dqo", "dko", "dq", "dk", "dqw", "dkw"):
        assert qk_bwd(L, **{name: P(13, 8)}) == ALIGN, name
    for out in ("dq", "dk", "dqw", "dkw", "ws"):
        for at in range(8):
            assert qk_bwd(L, **{out: P(at)}) == ALIAS, (out, at)
    assert qk_bwd(L, dq=P(9)) == ALIAS and qk_bwd(L, dqw=P(11, 16)) == ALIAS
    assert qk_bwd(L, ws=P(8)) == ALIAS
    assert qk_bwd(L, it=7) == DTYPE and qk_bwd(L, dim=12, rot=0) == UNSUP
    assert qk_bwd(L, rot=130) == SHAPE
    f = binding.ssm_qk_norm_rope_bwd_workspace_bytes
    assert f(-1, 1, 1, 64) == 0 and f(1, 1, 1, 12) == 0 and f(1, 1, 1, 264) == 0


DELTA = dict(q=P(0), k=P(1), v=P(2), qs=128, ks=128, vs=256, g=P(3), beta=P(4), h0=P(5), y=P(6),
             h1=P(7), kept=P(8), b=2, n=100, h=4, groups=2, dk=64, dv=64, it=1, gt=0, ot=1, ws=P(9),
             nw=1 << 29)


def delta(L, **kw):
    return L.ssm_gated_delta_fwd(*dict(DELTA, **kw).values(), None)


def test_delta(L):
    for name in ("q", "k", "v", "g", "beta", "y"):
        assert delta(L, **{name: None}) == NULL, name
    for name in ("b", "n", "h", "groups"):
        assert delta(L, **{name: -1}) == SHAPE, name
    assert delta(L, dk=0) == SHAPE and delta(L, dv=0) == SHAPE
    assert delta(L, groups=3) == SHAPE and delta(L, groups=0) == SHAPE and delta(L, h=0) == SHAPE
    assert delta(L, qs=127) == SHAPE and delta(L, ks=120) == SHAPE and delta(L, vs=255) == SHAPE
    assert delta(L, it=2) == DTYPE and delta(L, gt=-1) == DTYPE and delta(L, ot=9) == DTYPE
    assert delta(L, dk=60) == UNSUP and delta(L, dv=12) == UNSUP
    assert delta(L, dk=136, qs=272, ks=272) == UNSUP and delta(L, dv=264, vs=1056) == UNSUP
    assert delta(L, it=0) == UNSUP              # fp32 keeps nothing
    assert delta(L, n=1 << 30) == UNSUP and delta(L, b=1 << 28, n=1 << 10) == UNSUP
    assert delta(L, ws=None) == WS and delta(L, nw=1023) == WS
    need = binding.ssm_gated_delta_workspace_bytes(2, 100, 4, 64, 64)
    assert delta(L, kept=None, nw=need - 1) == WS
    for name in ("q", "k", "v", "h0", "y", "h1", "kept", "ws"):
        assert delta(L, **{name: P(10, 8)}) == ALIGN, name
    assert delta(L, g=P(10, 2)) == ALIGN and delta(L, beta=P(10, 1), gt=1) == ALIGN
    assert delta(L, qs=132) == ALIGN and delta(L, vs=260) == ALIGN
    assert delta(L, it=0, kept=None, n=4, ks=130) == ALIGN
    for out in ("y", "h1", "kept", "ws"):
        for at in range(6):
            if (out, at) != ("h1", 5):          # the state in place
                assert delta(L, **{out: P(at)}) == ALIAS, (out, at)
    assert delta(L, h1=P(5, 64)) == ALIAS
    assert delta(L, y=P(7)) == ALIAS and delta(L, kept=P(6)) == ALIAS and delta(L, ws=P(8, 16)) == ALIAS
    assert delta(L, b=0, q=None) == OK and delta(L, h=0, groups=0, q=None) == OK
    assert delta(L, n=0, q=None, h1=None) == OK and delta(L, n=0, q=None, h1=P(5)) == OK


DELTA_BWD = dict(q=P(0), k=P(1), v=P(2), qs=128, ks=128, vs=256, g=P(3), beta=P(4), h0=P(5),
                 dy=P(6), dlast=P(7), kept=P(8), dq=P(9), dk_=P(10), dv_=P(11), dg=P(12),
                 db=P(13), dh0=P(14), b=2, n=100, h=4, groups=2, dk=64, dv=64, it=1, gt=0, ot=1,
                 ws=P(15), nw=1 << 29)


def delta_bwd(L, **kw):
    return L.ssm_gated_delta_bwd(*dict(DELTA_BWD, **kw).values(), None)


def test_delta_bwd(L):
    for name in ("q", "k", "v", "g", "beta", "dy", "dq", "dk_", "dv_", "dg", "db"):
        assert delta_bwd(L, **{name: None}) == NULL, name
    assert delta_bwd(L, it=0) == UNSUP and delta_bwd(L, it=3) == DTYPE
    assert delta_bwd(L, dk=4) == UNSUP and delta_bwd(L, n=-1) == SHAPE
    assert delta_bwd(L, h=0) == SHAPE
    own = binding.ssm_gated_delta_bwd_workspace_bytes(2, 100, 4, 64, 64)
    kept = binding.ssm_gated_delta_checkpoint_bytes(2, 100, 4, 64, 64)
    assert delta_bwd(L, ws=None) == WS and delta_bwd(L, nw=own - 1) == WS
    assert delta_bwd(L, kept=None, nw=own + kept - 1) == WS
    for name in ("q", "k", "v", "h0", "dy", "dlast", "kept", "dq", "dk_", "dv_", "dh0", "ws"):
        assert delta_bwd(L, **{name: P(16, 8)}) == ALIGN, name
    for name in ("g", "beta", "dg", "db"):
        assert delta_bwd(L, **{name: P(16, 2)}) == ALIGN, name
    for i, out in enumerate(("dq", "dk_", "dv_", "dg", "db", "dh0", "ws")):
        for at in range(9):
            if (out, at) != ("dh0", 7):         # the state's gradient in place
                assert delta_bwd(L, **{out: P(at)}) == ALIAS, (out, at)
        other = 9 + (i + 1) % 7
        assert delta_bwd(L, **{out: P(other)}) == ALIAS, (out, other)
    assert delta_bwd(L, b=0, q=None) == OK
    assert delta_bwd(L, n=0, q=None, dh0=None) == OK


def test_delta_sizes(L):
    for f in (binding.ssm_gated_delta_checkpoint_bytes, binding.ssm_gated_delta_workspace_bytes,
              binding.ssm_gated_delta_bwd_workspace_bytes):
        assert f(1, 100, 4, 64, 64) > 0
        for bad in ((-1, 8, 4, 64, 64), (1, -8, 4, 64, 64), (1, 8, -4, 64, 64), (1, 8, 4, 60, 64),
                    (1, 8, 4, 64, 264), (1, 8, 4, 136, 64), (1, 8, 4, 0, 64), (1, 1 << 30, 4, 64, 64)):
            assert f(*bad) == 0, bad


def z(*shape, dt=BF16):
    return torch.zeros(*shape, dtype=dt)


def test_the_binding_takes_cuda_tensors_only():
    with pytest.raises(TypeError, match="CUDA"):
        binding.ssm_qk_norm_rope_fwd(z(1, 2, 3, 64))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        binding.ssm_qk_norm_rope_fwd(z(1, 2, 3, 64, dt=torch.float16))
    with pytest.raises(ValueError, match="4 dims"):
        binding.ssm_qk_norm_rope_fwd(z(2, 3, 64))
    five = z(1, 2, 2, 64), z(1, 2, 2, 64), z(1, 2, 4, 64), z(1, 2, 4), z(1, 2, 4)
    with pytest.raises(TypeError, match="CUDA"):
        binding.ssm_gated_delta_fwd(*five)
    with pytest.raises(TypeError, match="CUDA"):
        binding.ssm_gated_delta_bwd(*five, z(1, 2, 4, 64))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        binding.ssm_gated_delta_fwd(five[0].to(torch.float16), *five[1:])
    with pytest.raises(ValueError, match="multiple of ngroups"):
        binding.ssm_gated_delta_fwd(*five[:2], z(1, 2, 3, 64), *five[3:])
    with pytest.raises(ValueError, match="multiple of ngroups"):
        binding.ssm_gated_delta_fwd(*five[:2], z(1, 2, 0, 64), *five[3:])


def test_steps_between_tokens():
    """What _token_step takes, on CPU strides seen through a stand-in."""
    class Fake(torch.Tensor):
        is_cuda = True

    def step(t, shape=None):
        t = t.as_subclass(Fake)
        return binding._token_step(t, "t", t.dtype, shape or t.shape)

    wide = z(3, 5, 100)
    assert step(z(3, 5, 2, 8)) == 16
    assert step(wide[..., 8:24].unflatten(-1, (2, 8))) == 100
    assert step(wide[:, :1, 8:24].unflatten(-1, (2, 8))) == 500      # one token of each sequence
    assert step(wide[:1, :3, 8:24].unflatten(-1, (2, 8))) == 100     # a part of one sequence
    assert step(wide[:1, :1, 8:24].unflatten(-1, (2, 8))) == 16      # (contiguous as it is)
    for bad in (wide[:, :3, 8:24].unflatten(-1, (2, 8)), z(3, 5, 8, 2).transpose(2, 3),
                z(3, 2, 5, 8).transpose(1, 2), z(5, 3, 2, 8).transpose(0, 1),
                z(1, 1, 2, 8).expand(3, 5, 2, 8), wide[..., :32].unflatten(-1, (2, 16))[..., :8]):
        with pytest.raises(ValueError):
            step(bad)
    with pytest.raises(ValueError, match="shape"):
        step(z(3, 5, 2, 8), (3, 5, 4, 8))


def test_another_device_is_refused(monkeypatch):
    class On:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    monkeypatch.setattr(binding, "_devices", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    binding._one_device(On(0), On(0), None)
    with pytest.raises(ValueError, match="one device"):
        binding._one_device(On(0), None, On(1))
    with pytest.raises(ValueError, match="not the current one"):
        binding._one_device(On(1), On(1))
