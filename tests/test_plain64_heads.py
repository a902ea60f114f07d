"""The plain forms the query and key head operators are tested against: their gradients
against central differences."""
import numpy as np
import pytest

from tests import plain64_heads as H


def differences(f, x, d=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += d
        down[i] -= d
        g[i] = (f(up) - f(down)) / (2 * d)
    return g


@pytest.mark.parametrize("rot,inter", [(0, False), (6, False), (8, True), (4, True)])
def test_qk_gradient(rot, inter):
    rng = np.random.default_rng(rot)
    x, dy = rng.standard_normal((2, 3, 2, 8)), rng.standard_normal((2, 3, 2, 8))
    w = 1 + 0.2 * rng.standard_normal(8)
    phase = H.angles(rng.integers(0, 999, (2, 3)), 10.0 ** -np.arange(rot // 2)) if rot else None
    dx, dw = H.qk_bwd(x, w, phase, rot, 1e-3, dy, inter)

    def loss(x, w):
        return np.sum(dy * H.qk_fwd(x, w, phase, rot, 1e-3, inter))

    # central differences of a smooth function: 1e-12 of curvature, 1e-10 of rounding
    np.testing.assert_allclose(dx, differences(lambda v: loss(v, w), x), atol=1e-7)
    np.testing.assert_allclose(dw, differences(lambda v: loss(x, v), w), atol=1e-7)


def test_rotation_is_one():
    """Turning keeps lengths, is undone by turning back, and at two positions gives products
    that depend on their difference alone."""
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((2, 1, 1, 1, 16))
    f = 100.0 ** -np.arange(0, 1, 1 / 6)

    def at(v, p):
        return H.turn(v, H.angles(np.array([[p]]), f), 12, False)

    assert np.allclose(np.sum(at(x, 77) ** 2), np.sum(x ** 2))
    assert np.allclose(H.turn(at(x, 77), H.angles(np.array([[77]]), f), 12, False, back=True), x)
    assert np.allclose(np.sum(at(x, 5) * at(y, 9)), np.sum(at(x, 1005) * at(y, 1009)))


@pytest.mark.parametrize("groups,state", [(1, True), (2, True), (2, False)])
def test_delta_gradient(groups, state):
    rng = np.random.default_rng(groups)
    b, n, h, dk, dv = 1, 4, 2, 3, 2
    q, k = rng.standard_normal((2, b, n, groups, dk))
    v, dy = rng.standard_normal((2, b, n, h, dv))
    g, beta = -rng.random((b, n, h)), rng.random((b, n, h))
    S, dS = rng.standard_normal((2, b, h, dv, dk))
    if not state:
        S = dS = None

    def loss(**kw):
        a = dict(q=q, k=k, v=v, g=g, beta=beta, state=S)
        a.update(kw)
        y, last, _ = H.delta_fwd(**a)
        return np.sum(y * dy) + (np.sum(last * dS) if state else 0.0)

    grads = H.delta_bwd(q, k, v, g, beta, dy, S, dS)
    for name, x, got in zip(("q", "k", "v", "g", "beta", "state"), (q, k, v, g, beta, S), grads):
        if x is not None:
            ref = differences(lambda t: loss(**{name: t}), x)
            np.testing.assert_allclose(got, ref, atol=2e-7, err_msg=name)


def test_delta_masks():
    """A step with beta 0 is not looked at; a gate of -inf forgets whatever there was."""
    rng = np.random.default_rng(5)
    q, k = rng.standard_normal((2, 1, 6, 1, 4))
    v = rng.standard_normal((1, 6, 1, 3))
    g, beta = -rng.random((1, 6, 1)), rng.random((1, 6, 1))
    beta[0, 2] = 0
    k[0, 2], v[0, 2] = np.nan, np.nan
    y, last, _ = H.delta_fwd(q, k, v, g, beta)
    assert np.isfinite(y).all()
    grads = H.delta_bwd(q, k, v, g, beta, np.ones_like(v))
    assert all(np.isfinite(t).all() for t in grads[:5])
    assert not grads[1][0, 2].any() and not grads[2][0, 2].any() and not grads[4][0, 2].any()
    g[0, 4] = -np.inf
    y1, last1, _ = H.delta_fwd(q, k, v, g, beta)
    y2, last2, _ = H.delta_fwd(q[:, 4:], k[:, 4:], v[:, 4:], g[:, 4:], beta[:, 4:])
    assert np.array_equal(y1[:, 4:], y2) and np.array_equal(last1, last2)
    assert not H.delta_bwd(q, k, v, g, beta, np.ones_like(v))[3][0, 4].any()
