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
