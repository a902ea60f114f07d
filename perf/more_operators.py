"""The gated delta rule and what prepares its queries and keys, as measured cases: each
in a plain form (elementary torch operations) and through the library's entry points.

* qk:    RMS norm of every query and key head over its own columns, and the rotation
         by position, in one pass (``ssm_qk_norm_rope_fwd``), and its gradient
         (``ssm_qk_norm_rope_bwd``).
* delta: the gated delta rule  S = exp(g) S;  u = beta (v - S k);  S += u k^T;
         y = S q  per head (``ssm_gated_delta_fwd``: long sequences in chunks, a few
         tokens step by step), and its gradient (``ssm_gated_delta_bwd``).

``own`` chooses between the two forms; ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's queries and keys for a batch of 32 sequences: latency
        {"name": "qk step", "op": "qk", "batch": 32, "seqlen": 1, "qheads": 32, "kheads": 8,
         "dim": 128, "rot": 128, "pairs": "halves", "type": "bf16", "packed": True, "far": True},
        # a prefill of 16384 tokens far into a document; half of each head is rotated
        {"name": "qk prefill", "op": "qk", "batch": 1, "seqlen": 16384, "qheads": 32,
         "kheads": 8, "dim": 128, "rot": 64, "pairs": "halves", "type": "bf16", "packed": True,
         "far": True},
        # a training step, queries and keys ranges of one projection
        {"name": "qk train", "op": "qk_train", "batch": 8, "seqlen": 2048, "qheads": 16,
         "kheads": 16, "dim": 128, "rot": 128, "pairs": "halves", "type": "bf16",
         "packed": True, "far": False},
        # odd sizes in 32 bits, neighbouring columns rotated
        {"name": "qk train odd", "op": "qk_train", "batch": 3, "seqlen": 1021, "qheads": 7,
         "kheads": 3, "dim": 72, "rot": 20, "pairs": "neighbours", "type": "f32",
         "packed": False, "far": False},
        # one token of one sequence: latency
        {"name": "delta step one", "op": "delta", "batch": 1, "seqlen": 1, "heads": 32,
         "groups": 16, "dk": 128, "dv": 128, "type": "bf16", "gates": "f32", "state": True,
         "packed": True, "padded": False},
        # one token for 256 sequences: bound by reading and writing the states
        {"name": "delta step", "op": "delta", "batch": 256, "seqlen": 1, "heads": 32,
         "groups": 32, "dk": 128, "dv": 64, "type": "bf16", "gates": "f32", "state": True,
         "packed": True, "padded": False},
        # six drafted tokens in 32 bits, resumed from the states
        {"name": "delta drafted", "op": "delta", "batch": 16, "seqlen": 6, "heads": 16,
         "groups": 16, "dk": 128, "dv": 128, "type": "f32", "gates": "f32", "state": True,
         "packed": False, "padded": False},
        # prefill of a batch of short prompts, padded to one length
        {"name": "delta prefill", "op": "delta", "batch": 32, "seqlen": 256, "heads": 32,
         "groups": 32, "dk": 128, "dv": 64, "type": "bf16", "gates": "f32", "state": False,
         "packed": True, "padded": True},
        # the prefill of one long document: few heads, many steps
        {"name": "delta long", "op": "delta", "batch": 1, "seqlen": 32768, "heads": 16,
         "groups": 16, "dk": 128, "dv": 128, "type": "bf16", "gates": "f32", "state": False,
         "packed": True, "padded": False},
        # a training step on packed documents
        {"name": "delta train", "op": "delta_train", "batch": 8, "seqlen": 2048, "heads": 16,
         "groups": 16, "dk": 128, "dv": 128, "type": "bf16", "gates": "bf16", "state": False,
         "packed": True, "padded": False},
        # odd sizes, shared key heads, resumed from a state, padded
        {"name": "delta train odd", "op": "delta_train", "batch": 3, "seqlen": 1021, "heads": 6,
         "groups": 2, "dk": 72, "dv": 40, "type": "bf16", "gates": "bf16", "state": True,
         "packed": False, "padded": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "qk_train", "delta", "delta", "delta_train"])
    batch, seqlen = _log_int(rng, 1, 256), _log_int(rng, 1, 32768)
    if op.startswith("qk"):
        dim = rng.choice([64, 128, 256, 8 * rng.randint(2, 32)])
        case = {"op": op, "qheads": rng.randint(1, 32), "kheads": rng.randint(1, 16), "dim": dim,
                "rot": rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2), 0]),
                "pairs": rng.choice(["halves", "neighbours"]),
                "type": rng.choice(["bf16", "bf16", "f32"]), "packed": rng.random() < 0.5,
                "far": rng.random() < 0.5}
        most = 16384 * 40 * 128 // (1 if op == "qk" else 2)
        row = (case["qheads"] + case["kheads"]) * dim
    else:
        heads = _log_int(rng, 1, 32)
        case = {"op": op, "heads": heads,
                "groups": rng.choice([g for g in range(1, heads + 1) if heads % g == 0]),
                "dk": rng.choice([64, 128, 8 * rng.randint(2, 16)]),
                "dv": rng.choice([64, 128, 8 * rng.randint(2, 16)]),
                "type": "bf16", "gates": "bf16" if op == "delta_train" else "f32",
                "state": rng.random() < 0.5, "packed": rng.random() < 0.5}
        if op == "delta" and rng.random() < 0.3:
            case["type"], seqlen = "f32", min(seqlen, 16)
        case["padded"] = seqlen > 16 and rng.random() < 0.3
        most = 32768 * 16 * 128 // (1 if op == "delta" else 2)
        row = heads * max(case["dk"], case["dv"])
        batch = max(1, min(batch, 256 * 32 * 64 * 128 // (heads * case["dk"] * case["dv"])))
    seqlen = max(1, min(seqlen, most // row))
    case["batch"], case["seqlen"] = max(1, min(batch, most // (row * seqlen))), seqlen
    return case


def work(case):
    b, n, e = case["batch"], case["seqlen"], _SIZE[case["type"]]
    if case["op"].startswith("qk"):
        values = b * n * (case["qheads"] + case["kheads"]) * case["dim"]
        once = 8 * b * n + 8 * case["dim"] + 4 * case["rot"]    # positions, weights, frequencies
        if case["op"] == "qk":
            return {"bytes": 2 * values * e + once, "flops": 8 * values}
        return {"bytes": 4 * values * e + once + 8 * case["dim"], "flops": 26 * values}
    h, dk, dv = case["heads"], case["dk"], case["dv"]
    qk, v, gates = b * n * case["groups"] * dk * e, b * n * h * dv * e, b * n * h
    states = 4 * b * h * dk * dv
    fwd = 2 * qk + 2 * v + 2 * gates * _SIZE[case["gates"]] + states * (2 if case["state"] else 1)
    flops = 7 * gates * dk * dv
    if case["op"] == "delta":
        return {"bytes": fwd, "flops": flops}
    # dy, then the gradients of q, k, v and both gates, the final state's gradient and
    # the initial state's
    more = 2 * qk + 2 * v + 2 * gates * _SIZE[case["gates"]] + (2 * states if case["state"] else 0)
    return {"bytes": fwd + more, "flops": 3 * flops}


# ------------------------------------------------------------------ inputs

def _ranges(parts, dims, packed):
    """parts (batch, seqlen, heads, dim): each by itself, or column ranges of one
    projection with further columns behind them."""
    if not packed:
        return parts
    b, n = parts[0].shape[:2]
    flat = [p.reshape(b, n, -1) for p in parts]
    whole = torch.cat(flat + [torch.zeros_like(flat[0][..., :8])], -1)
    got, at = [], 0
    for p, (heads, dim) in zip(flat, dims):
        got.append(whole[..., at:at + heads * dim].unflatten(-1, (heads, dim)))
        at += heads * dim
    return got


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    b, n, td = case["batch"], case["seqlen"], _TYPES[case["type"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"].startswith("qk"):
        d, rot = case["dim"], case["rot"]
        dims = [(case["qheads"], d), (case["kheads"], d)]
        # heads of different sizes, as projections give them
        parts = [(randn(b, n, h, d) * torch.exp(randn(h, 1))).to(td) for h, _ in dims]
        s["q"], s["k"] = _ranges(parts, dims, case["packed"])
        s["wq"], s["wk"] = 1 + 0.1 * randn(d), 1 + 0.1 * randn(d)
        first = torch.randint(1 << 20 if case["far"] else 1, (b, 1), generator=g, device="cuda")
        s["positions"] = first + torch.arange(n, device="cuda")
        s["freq"] = None
        if rot:
            at = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
            s["freq"] = 10000.0 ** (-2 * at / rot)
        if case["op"] == "qk_train":
            s["dq"], s["dk"] = (randn(b, n, h, d).to(td) for h, _ in dims)
        return s
    h, groups, dk, dv = case["heads"], case["groups"], case["dk"], case["dv"]
    unit = torch.nn.functional.normalize
    # queries and keys of length one, as the norms leave them; keys share a direction
    s["q"] = unit(randn(b, n, groups, dk), dim=-1).to(td)
    s["k"] = unit(randn(b, n, groups, dk) + 0.3 * randn(1, 1, groups, dk), dim=-1).to(td)
    s["v"], = _ranges([randn(b, n, h, dv).to(td)], [(h, dv)], case["packed"])
    # heads that forget within a few steps and within thousands
    rate = torch.exp(-6 * rand(h))
    gate = -rate * torch.nn.functional.softplus(randn(b, n, h))
    beta = torch.sigmoid(randn(b, n, h))
    if n > 64:
        # documents packed one after another: the first token starts the state anew
        gate = gate.masked_fill(rand(b, n, 1) < 1.0 / 512, float("-inf"))
    if case["padded"]:
        # behind a sequence's end nothing is forgotten and nothing learned
        ends = 1 + (rand(b, 1, 1) * n).long()
        behind = torch.arange(n, device="cuda")[None, :, None] >= ends
        gate, beta = gate.masked_fill(behind, 0.0), beta.masked_fill(behind, 0.0)
    s["g"], s["beta"] = gate.to(_TYPES[case["gates"]]), beta.to(_TYPES[case["gates"]])
    s["state"] = randn(b, h, dv, dk) / math.sqrt(dk) if case["state"] else None
    if case["op"] == "delta_train":
        s["dy"] = randn(b, n, h, dv).to(td)
        s["dfinal"] = randn(b, h, dv, dk) if case["state"] else None
    return s


# -------------------------------------------------------------------- run

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import state_space_model_selective_gb300 as ssm

    case = s["case"]
    if case["op"].startswith("qk"):
        args = dict(q_weight=s["wq"], k_weight=s["wk"], positions=s["positions"],
                    inv_freq=s["freq"], eps=EPS, interleaved=case["pairs"] == "neighbours")
        q, k = ssm.ssm_qk_norm_rope_fwd(s["q"], s["k"], **args)
        if case["op"] == "qk":
            return {"q": q, "k": k}
        g = ssm.ssm_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], **args)
        return {"q": q, "k": k, "dq": g["dq"], "dk": g["dk"], "dwq": g["dq_weight"],
                "dwk": g["dk_weight"]}
    kept = None
    if case["op"] == "delta_train":
        size = ssm.ssm_gated_delta_checkpoint_bytes(case["batch"], case["seqlen"], case["heads"],
                                                    case["dk"], case["dv"])
        kept = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
    y, final = ssm.ssm_gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"],
                                       initial_state=s["state"], checkpoints=kept)
    if case["op"] == "delta":
        return {"y": y, "final": final}
    g = ssm.ssm_gated_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"],
                                initial_state=s["state"], dfinal_state=s["dfinal"],
                                checkpoints=kept, want_dinitial_state=s["state"] is not None)
    return {"y": y, "final": final, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"], "dg": g["dg"],
            "dbeta": g["dbeta"], "dstate": g["dinitial_state"]}


def _plain(s):
    return _plain_qk(s) if s["case"]["op"].startswith("qk") else _plain_delta(s)


def _turn(x, cos, sin, rot, pairs, back=False):
    """x's first rot columns turned by each pair's angle, or turned back."""
    if not rot:
        return x
    if pairs == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    if back:
        sin = -sin
    c, d = a * cos - b * sin, a * sin + b * cos
    both = torch.cat([c, d], -1) if pairs == "halves" else torch.stack([c, d], -1).flatten(-2)
    return torch.cat([both, x[..., rot:]], -1)


def _plain_qk(s):
    case = s["case"]
    rot, pairs, td = case["rot"], case["pairs"], s["q"].dtype
    cos = sin = None
    if rot:
        # far positions' angles in 64 bits
        angle = (s["positions"].double()[..., None] * s["freq"])[:, :, None]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def forward(x, w):
        x = x.float()
        n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return _turn(n * w, cos, sin, rot, pairs).to(td)

    def backward(x, w, dy):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n, dy = x * r, _turn(dy.float(), cos, sin, rot, pairs, back=True)
        gw = dy * w
        return (r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(td), (dy * n).sum((0, 1, 2))

    out = {"q": forward(s["q"], s["wq"]), "k": forward(s["k"], s["wk"])}
    if case["op"] == "qk_train":
        out["dq"], out["dwq"] = backward(s["q"], s["wq"], s["dq"])
        out["dk"], out["dwk"] = backward(s["k"], s["wk"], s["dk"])
    return out


CHUNK = 64


def _chunks(x, chunks):
    """(batch, seqlen, heads, ...) to (chunks, batch, heads, CHUNK, ...), zeros behind."""
    b, n, h = x.shape[:3]
    pad = chunks * CHUNK - n
    if pad:
        x = torch.cat([x, x.new_zeros(b, pad, *x.shape[2:])], 1)
    x = x.reshape(b, chunks, CHUNK, h, *x.shape[3:])
    return x.transpose(2, 3).transpose(0, 1)


def _delta_chunked(q, k, v, g, beta, state):
    """The delta rule in 32 bits, chunk by chunk: within a chunk the steps' updates U
    solve (1 + A) U = beta (V - decay K S)."""
    b, n, h, dv = v.shape
    ratio, chunks = h // q.shape[2], -(-n // CHUNK)
    q, k = q.repeat_interleave(ratio, 2), k.repeat_interleave(ratio, 2)
    learns = (beta != 0)[..., None]
    k, v = torch.where(learns, k, 0.0), torch.where(learns, v, 0.0)
    q, k, v, g, beta = (_chunks(x, chunks) for x in (q, k, v, g, beta))
    # sums of logarithms in 64 bits: what a far one leaves cancels in the differences
    total = g.double().clamp(min=-1000.0).cumsum(-1)
    decay = torch.exp((total[..., :, None] - total[..., None, :]).clamp(max=700.0)).float().tril()
    into = torch.exp(total).float()[..., None]                 # from the chunk's start
    out = torch.exp(total[..., -1:] - total).float()[..., None]  # to its end
    whole = into[..., -1:, :]
    kk, qk = k @ k.transpose(-1, -2), q @ k.transpose(-1, -2)
    power = -(beta[..., None] * kk * decay).tril(-1)
    eye = torch.eye(CHUNK, device=v.device)
    solve = eye + power
    for _ in range(5):      # (1 - P)^-1 = (1 + P)(1 + P^2)(1 + P^4) ...: P^64 = 0
        power = power @ power
        solve = solve @ (eye + power)
    attend, ys = qk * decay, []
    for c in range(chunks):
        u = solve[c] @ (beta[c][..., None] * (v[c] - into[c] * (k[c] @ state)))
        ys.append(into[c] * (q[c] @ state) + attend[c] @ u)
        state = whole[c] * state + (k[c] * out[c]).transpose(-1, -2) @ u
    y = torch.stack(ys, 1).transpose(2, 3).reshape(b, chunks * CHUNK, h, dv)[:, :n]
    return y, state


def _plain_delta(s):
    case, td = s["case"], s["q"].dtype
    b, n, h, dv = s["v"].shape
    train = case["op"] == "delta_train"
    ins = [s[x].float().detach() for x in ("q", "k", "v", "g", "beta")]
    state = s["state"]
    state = (torch.zeros(b, h, dv, case["dk"], device=s["v"].device) if state is None
             else state.detach().clone())
    if n == 1:
        # one step as it is defined
        q, k, v, g, beta = (x[:, 0] for x in ins)
        q, k = (x.repeat_interleave(h // case["groups"], 1) for x in (q, k))
        learns = (beta != 0)[..., None]
        k, v = torch.where(learns, k, 0.0), torch.where(learns, v, 0.0)
        if not train:
            state = state * torch.exp(g)[..., None, None]
            u = beta[..., None] * (v - (state * k[..., None, :]).sum(-1))
            state = state + u[..., None] * k[..., None, :]
            return {"y": (state * q[..., None, :]).sum(-1)[:, None].to(td), "final": state}
    if not train:
        y, state = _delta_chunked(*ins, state.transpose(-1, -2))
        return {"y": y.to(td), "final": state.transpose(-1, -2).contiguous()}
    with torch.enable_grad():
        leaves = [x.requires_grad_() for x in ins + [state]]
        y, final = _delta_chunked(*leaves[:5], leaves[5].transpose(-1, -2))
        final = final.transpose(-1, -2)
        loss = (y * s["dy"].float()).sum()
        if s["dfinal"] is not None:
            loss = loss + (final * s["dfinal"]).sum()
        dq, dk, dv_, dg, dbeta, dstate = torch.autograd.grad(loss, leaves)
    # a step that learns nothing (beta 0) is masked: its key, value and beta have no part
    dbeta = torch.where(ins[4] == 0, 0.0, dbeta)
    dg = torch.where(torch.exp(ins[3]) == 0, 0.0, dg)
    gt = s["g"].dtype
    return {"y": y.detach().to(td), "final": final.detach().contiguous(), "dq": dq.to(td),
            "dk": dk.to(td), "dv": dv_.to(td), "dg": dg.to(gt), "dbeta": dbeta.to(gt),
            "dstate": None if s["state"] is None else dstate}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definition in 64 bits: the norm's gradient from the quotient's derivative,
    rotations as complex products, the delta rule and its adjoint step by step."""
    s = prepare(case, seed)
    return _exact_qk(s) if case["op"].startswith("qk") else _exact_delta(s)


def _exact_qk(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    out = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x, w = s[name].double(), w.double()
        d = x.shape[-1]
        rms = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
        first, second = ((torch.arange(half), torch.arange(half) + half)
                         if case["pairs"] == "halves"
                         else (2 * torch.arange(half), 2 * torch.arange(half) + 1))
        y = x / rms * w
        if rot:
            phase = torch.outer(s["positions"].reshape(-1).double(), s["freq"])
            turn = torch.polar(torch.ones_like(phase), phase).reshape(*x.shape[:2], 1, half)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
        if case["op"] == "qk_train":
            dy = s["d" + name].double()
            if rot:
                z = torch.complex(dy[..., first], dy[..., second]) * turn.conj()
                dy[..., first], dy[..., second] = z.real, z.imag
            dn = dy * w
            out["d" + name] = dn / rms - x * (dn * x).sum(-1, keepdim=True) / (d * rms ** 3)
            out["dw" + name] = (dy * x / rms).sum((0, 1, 2))
    return out


def _exact_delta(s):
    case = s["case"]
    b, n, h, dv = s["v"].shape
    groups, dk, span = case["groups"], case["dk"], 128
    if n * b * h * dk * dv > 40 * 2048 * 64 * 128 * 128:
        return None

    def heads(x):
        return x.double().repeat_interleave(h // groups, 2)

    q, k, v, a, beta = (heads(s["q"]), heads(s["k"]), s["v"].double(), s["g"].double().exp(),
                        s["beta"].double())
    k, v = k * (beta != 0)[..., None], v * (beta != 0)[..., None]
    state = torch.zeros(b, h, dv, dk, dtype=torch.float64, device=v.device)
    if s["state"] is not None:
        state = s["state"].double()

    def step(state, t):
        state = state * a[:, t, :, None, None]
        error = v[:, t] - torch.einsum("bhvk,bhk->bhv", state, k[:, t])
        new = torch.einsum("bhv,bhk->bhvk", beta[:, t, :, None] * error, k[:, t])
        return new.add_(state), error

    kept, y = [], torch.empty_like(v)
    for t in range(n):
        if t % span == 0:
            kept.append(state)
        state, _ = step(state, t)
        y[:, t] = torch.einsum("bhvk,bhk->bhv", state, q[:, t])
    out = {"y": y, "final": state}
    if case["op"] == "delta":
        return out
    dy = s["dy"].double()
    lam = torch.zeros_like(state) if s["dfinal"] is None else s["dfinal"].double()
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(a), torch.empty_like(beta)
    for first in range((n - 1) // span * span, -1, -span):
        before, errors = [kept[first // span]], []
        for t in range(first, min(n, first + span)):
            after, error = step(before[-1], t)
            before.append(after)
            errors.append(error)
        for t in range(min(n, first + span) - 1, first - 1, -1):
            old, new, error = before[t - first], before[t - first + 1], errors[t - first]
            dq[:, t] = torch.einsum("bhvk,bhv->bhk", new, dy[:, t])
            lam = lam + torch.einsum("bhv,bhk->bhvk", dy[:, t], q[:, t])
            du = torch.einsum("bhvk,bhk->bhv", lam, k[:, t])
            dbeta[:, t] = (du * error).sum(-1)
            dv_[:, t] = du * beta[:, t, :, None]
            decayed = old * a[:, t, :, None, None]
            dk_[:, t] = (torch.einsum("bhvk,bhv->bhk", lam, beta[:, t, :, None] * error)
                         - torch.einsum("bhvk,bhv->bhk", decayed, dv_[:, t]))
            lam = lam - torch.einsum("bhv,bhk->bhvk", dv_[:, t], k[:, t])
            dg[:, t] = (lam * decayed).sum((-1, -2))
            lam = lam * a[:, t, :, None, None]
    off = beta == 0
    shared = (b, n, groups, h // groups, dk)
    out.update(dq=dq.reshape(shared).sum(3),
               dk=dk_.masked_fill(off[..., None], 0.0).reshape(shared).sum(3), dv=dv_, dg=dg,
               dbeta=dbeta.masked_fill(off, 0.0), dstate=None if s["state"] is None else lam)
    return out
