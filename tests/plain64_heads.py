"""Plain 64-bit implementations of the operators on query and key heads (norm with the
rotation by position, gated delta rule), forward and gradient, in numpy: the references
of their GPU tests.  Their gradients are checked against differences in
test_plain64_heads.py."""
import numpy as np


# ------------------------------------------------- norm and rotation of heads

def pairs_of(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def angles(positions, inv_freq):
    """(batch, seqlen, 1, rot / 2): whole turns are taken off in 80 bits."""
    turns = positions.astype(np.longdouble)[..., None] * (
        inv_freq.astype(np.longdouble) / (2 * np.longdouble(np.pi)))
    turns -= np.floor(turns)
    return (turns.astype(np.float64) * 2 * np.pi)[:, :, None]


def turn(x, phase, rot, interleaved, back=False):
    if not rot:
        return x
    a, b = pairs_of(rot, interleaved)
    c, s = np.cos(phase), np.sin(phase) * (-1 if back else 1)
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def qk_fwd(x, w, phase, rot, eps, interleaved=False):
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return turn(n if w is None else n * w, phase, rot, interleaved)


def qk_bwd(x, w, phase, rot, eps, dy, interleaved=False):
    """dx and dw."""
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n, g = x * r, turn(dy, phase, rot, interleaved, back=True)
    gw = g if w is None else g * w
    return r * (gw - n * np.mean(gw * n, -1, keepdims=True)), np.sum(g * n, (0, 1, 2))


# ------------------------------------------------------------ gated delta rule

def _to_heads(x, heads):
    return np.repeat(x, heads // x.shape[2], 2)


def delta_fwd(q, k, v, g, beta, state=None):
    """y, the final state and every state (batch, seqlen + 1, heads, headdim, dstate).  A step
    with beta 0 is masked: its key and value are not looked at."""
    b, n, h, dv = v.shape
    q, k = _to_heads(q, h), _to_heads(k, h)
    off = beta == 0
    k, v = np.where(off[..., None], 0.0, k), np.where(off[..., None], 0.0, v)
    S = np.zeros((b, h, dv, q.shape[3])) if state is None else state.astype(np.float64)
    y, kept = np.empty(v.shape), [S]
    for t in range(n):
        a = np.exp(g[:, t])[..., None, None]
        S = np.where(a == 0, 0.0, a * np.where(a == 0, 0.0, S))
        u = beta[:, t, :, None] * (v[:, t] - np.einsum("bhvk,bhk->bhv", S, k[:, t]))
        S = S + u[..., None] * k[:, t, :, None, :]
        y[:, t] = np.einsum("bhvk,bhk->bhv", S, q[:, t])
        kept.append(S)
    return y, S, np.stack(kept, 1)


def delta_bwd(q, k, v, g, beta, dy, state=None, dfinal=None):
    """dq, dk, dv, dg, dbeta, dstate; 0 for a masked step's k, v and beta."""
    b, n, h, dv_ = v.shape
    groups, dk_ = q.shape[2:]
    _, _, states = delta_fwd(q, k, v, g, beta, state)
    qh, kh = _to_heads(q, h), _to_heads(k, h)
    off = beta == 0
    kh, v = np.where(off[..., None], 0.0, kh), np.where(off[..., None], 0.0, v)
    L = np.zeros(states[:, 0].shape) if dfinal is None else dfinal.astype(np.float64)
    dq, dk, dv = np.empty(qh.shape), np.empty(qh.shape), np.empty(v.shape)
    dg, db = np.empty(g.shape), np.empty(g.shape)
    for t in range(n - 1, -1, -1):
        a = np.exp(g[:, t])[..., None, None]
        old = np.where(a == 0, 0.0, a * np.where(a == 0, 0.0, states[:, t]))  # decayed
        bt = beta[:, t, :, None]
        e = v[:, t] - np.einsum("bhvk,bhk->bhv", old, kh[:, t])
        dq[:, t] = np.einsum("bhvk,bhv->bhk", states[:, t + 1], dy[:, t])
        L = L + dy[:, t, :, :, None] * qh[:, t, :, None, :]
        du = np.einsum("bhvk,bhk->bhv", L, kh[:, t])
        db[:, t] = np.sum(du * e, -1)
        dv[:, t] = du * bt
        dk[:, t] = (np.einsum("bhvk,bhv->bhk", L, bt * e) -
                    np.einsum("bhvk,bhv->bhk", old, dv[:, t]))
        L = L - dv[:, t, :, :, None] * kh[:, t, :, None, :]
        dg[:, t] = np.sum(L * old, (-1, -2))
        L = a * L
    dk, db = np.where(off[..., None], 0.0, dk), np.where(off, 0.0, db)
    dq, dk = (x.reshape(b, n, groups, h // groups, dk_).sum(3) for x in (dq, dk))
    return dq, dk, dv, dg, db, L
