"""Plain 64-bit implementations of the operators around the mixers (norm,
gated recurrence, vocabulary cross entropy), forward and gradient, in numpy:
the references of their GPU tests.  Their gradients are themselves checked
against differences in test_plain64.py."""
import numpy as np

E4M3_MAX = 448.0


def sigmoid(v):
    out = np.empty_like(v)
    pos = v >= 0
    out[pos] = 1 / (1 + np.exp(-v[pos]))
    e = np.exp(v[~pos])
    out[~pos] = e / (1 + e)
    return out


def silu(z):
    return z * sigmoid(z)


# ------------------------------------------------------------------ norm

def norm_fwd(x, residual, weight, eps):
    s = x if residual is None else x + residual
    return s / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps) * weight, s


def norm_bwd(s, weight, eps, dy, dsum=None):
    r = 1 / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps)
    n, g = s * r, dy * weight
    d = r * (g - n * np.mean(g * n, -1, keepdims=True))
    return (d if dsum is None else d + dsum), np.sum(dy * n, 0)


def e4m3_round(v):
    """Nearest e4m3 value (ties to even), magnitudes above 448 to 448: the grid has
    3 mantissa bits from 2^-6 up and steps of 2^-9 below."""
    a = np.abs(v)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    ulp = 2.0 ** (np.maximum(e, -6) - 3)
    return np.sign(v) * np.minimum(np.rint(a / ulp) * ulp, E4M3_MAX)


def group_amax(y, group):
    """(rows, groups) largest magnitudes, the last group as long as what is left."""
    dim = y.shape[1]
    group = group or dim
    return np.stack([np.max(np.abs(y[:, c:c + group]), 1) for c in range(0, dim, group)], 1)


# ------------------------------------------------------------- recurrence

def linrec_fwd(f, x, z=None, h0=None):
    """Returns y, final state and every state h_t, (batch, seqlen, dim)."""
    batch, n, dim = x.shape
    h = np.zeros((batch, dim)) if h0 is None else h0.astype(np.float64)
    hs = np.empty((batch, n, dim))
    for t in range(n):
        a, om = sigmoid(f[:, t]), sigmoid(-f[:, t])
        kept = np.where(a == 0, 0.0, a * np.where(a == 0, 0.0, h))
        h = kept + np.where(om == 0, 0.0, om * np.where(om == 0, 0.0, x[:, t]))
        hs[:, t] = h
    return (hs if z is None else hs * silu(z)), h, hs


def linrec_bwd(f, x, dy, z=None, h0=None, dfinal=None):
    """df, dx, dz (None without z), dh0."""
    batch, n, dim = x.shape
    _, _, hs = linrec_fwd(f, x, None, h0)
    mu = np.zeros((batch, dim)) if dfinal is None else dfinal.astype(np.float64)
    df, dx = np.empty_like(hs), np.empty_like(hs)
    for t in range(n - 1, -1, -1):
        a, om = sigmoid(f[:, t]), sigmoid(-f[:, t])
        lam = mu + (dy[:, t] if z is None else dy[:, t] * silu(z[:, t]))
        before = hs[:, t - 1] if t else (np.zeros((batch, dim)) if h0 is None else h0)
        s = a * om
        xt = np.where(om == 0, 0.0, x[:, t])
        df[:, t] = np.where(s == 0, 0.0, lam * (np.where(s == 0, 0.0, before) - xt) * s)
        dx[:, t] = np.where(om == 0, 0.0, lam * om)
        mu = np.where(a == 0, 0.0, a * lam)
    dz = None
    if z is not None:
        sg = sigmoid(z)
        dz = dy * hs * (sg + z * sg * (1 - sg))
    return df, dx, dz, mu


# ---------------------------------------------------------- cross entropy

def ce_fwd(h, W, targets):
    """loss (0 where the target is negative) and log-sum-exp per token."""
    logits = h @ W.T
    m = logits.max(-1)
    lse = m + np.log(np.exp(logits - m[:, None]).sum(-1))
    rows = np.flatnonzero(targets >= 0)
    loss = np.zeros(len(h))
    loss[rows] = lse[rows] - logits[rows, targets[rows]]
    return loss, lse


def ce_bwd(h, W, targets, dloss):
    logits = h @ W.T
    p = np.exp(logits - ce_fwd(h, W, targets)[1][:, None])
    rows = np.flatnonzero(targets >= 0)
    p[rows, targets[rows]] -= 1
    p *= np.where(targets >= 0, dloss, 0.0)[:, None]
    return p @ W, p.T @ h
