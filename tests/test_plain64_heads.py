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
