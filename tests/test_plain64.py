"""The 64-bit references' gradients against central differences of their forwards,
and their masked steps against what the operators promise."""
import numpy as np
import pytest

from tests import plain64 as P


def _check(loss, params, grads, step=1e-6, tol=1e-7):
    """Every entry of every gradient against (L(p + e) - L(p - e)) / 2e: the error is
    the third derivative's step^2 and rounding's 1e-16 |L| / step, each below 1e-9 here."""
    for name, p in params.items():
        num = np.empty_like(p)
        for i in np.ndindex(p.shape):
            old = p[i]
            p[i] = old + step
            up = loss()
            p[i] = old - step
            num[i] = (up - loss()) / (2 * step)
            p[i] = old
        err = np.max(np.abs(num - grads[name])) / max(1.0, np.max(np.abs(num)))
        assert err < tol, (name, err)


@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradient(residual):
    g = np.random.default_rng(0)
    x, w, dy = g.normal(size=(3, 7)), g.normal(size=7), g.normal(size=(3, 7))
    res = g.normal(size=(3, 7)) if residual else None
    ds = g.normal(size=(3, 7))

    def loss():
        y, s = P.norm_fwd(x, res, w, 1e-3)
        return np.sum(dy * y) + np.sum(ds * s)

    dx, dw = P.norm_bwd(x if res is None else x + res, w, 1e-3, dy, ds)
    params, grads = {"x": x, "w": w}, {"x": dx, "w": dw}
    if residual:
        params["res"], grads["res"] = res, dx
    _check(loss, params, grads)


@pytest.mark.parametrize("gated,state", [(False, False), (True, False), (True, True)])
def test_linrec_gradient(gated, state):
    g = np.random.default_rng(1)
    shape = (2, 5, 3)
    f, x, dy = (g.normal(size=shape) for _ in range(3))
    z = g.normal(size=shape) if gated else None
    h0 = g.normal(size=(2, 3)) if state else None
    dfin = g.normal(size=(2, 3)) if state else None

    def loss():
        y, fin, _ = P.linrec_fwd(f, x, z, h0)
        return np.sum(dy * y) + (np.sum(dfin * fin) if state else 0.0)

    df, dx, dz, dh0 = P.linrec_bwd(f, x, dy, z, h0, dfin)
    params, grads = {"f": f, "x": x}, {"f": df, "x": dx}
    if gated:
        params["z"], grads["z"] = z, dz
    if state:
        params["h0"], grads["h0"] = h0, dh0
    _check(loss, params, grads)


def test_linrec_masked_steps():
    """A gate of +inf holds the state past a NaN input; -inf drops a NaN state."""
    f = np.array([0.0, np.inf, -np.inf, 1.0]).reshape(1, 4, 1)
    x = np.array([2.0, np.nan, 3.0, 1.0]).reshape(1, 4, 1)
    _, _, hs = P.linrec_fwd(f, x, None, np.array([[1.0]]))
    assert hs[0, 0, 0] == 1.5 and hs[0, 1, 0] == 1.5 and hs[0, 2, 0] == 3.0
    assert np.isfinite(P.linrec_fwd(f[:, 2:], x[:, 2:], None, np.array([[np.nan]]))[1]).all()
    df, dx, _, _ = P.linrec_bwd(f, x, np.ones((1, 4, 1)), None, np.array([[1.0]]))
    assert df[0, 1, 0] == 0 and df[0, 2, 0] == 0 and dx[0, 1, 0] == 0 and np.isfinite(df).all()


def test_cross_entropy_gradient():
    g = np.random.default_rng(2)
    h, W = g.normal(size=(4, 3)), g.normal(size=(6, 3))
    targets, dloss = np.array([5, -100, 0, 2]), g.uniform(0.1, 1, size=4)

    def loss():
        return np.sum(dloss * P.ce_fwd(h, W, targets)[0])

    dh, dW = P.ce_bwd(h, W, targets, dloss)
    _check(loss, {"h": h, "W": W}, {"h": dh, "W": dW})
    assert np.all(dh[1] == 0)


def test_e4m3_grid():
    v = np.array([0.0, 448.0, 500.0, -17.0, 2.0 ** -9, 2.0 ** -10, 1.0625, 1.1875, 0.3])
    want = np.array([0.0, 448.0, 448.0, -16.0, 2.0 ** -9, 0.0, 1.0, 1.25, 0.3125])
    np.testing.assert_array_equal(P.e4m3_round(v), want)
