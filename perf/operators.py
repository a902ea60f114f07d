"""The operators a recurrent language model needs around its scans, as measured
cases: each in a plain form (elementary torch operations in 32 bits) and through
the library's entry points.

* norm:   RMS norm with the residual's addition (``ssm_add_rmsnorm_fwd``), the
          same with an 8-bit output and scales (``ssm_add_rmsnorm_e4m3_fwd``),
          and its gradient (``ssm_add_rmsnorm_bwd``).
* linrec: the gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t with
          a_t = sigmoid(f_t) and the output gate y_t = h_t silu(z_t)
          (``ssm_linrec_fwd``), and its gradient (``ssm_linrec_bwd``).
* ce:     softmax cross entropy of h W^T over a large vocabulary without the
          logits in memory (``ssm_vocab_ce_fwd``), and its gradient
          (``ssm_vocab_ce_bwd``).

``own`` chooses between the two forms; ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's norm for a batch of 16 sequences: latency
        {"name": "norm step", "op": "norm", "rows": 16, "dim": 1536, "type": "bf16",
         "residual": "bf16"},
        # a prefill of 16384 tokens feeding an 8-bit product, scales per 128 columns
        {"name": "norm 8-bit prefill", "op": "norm_q8", "rows": 16384, "dim": 2048,
         "type": "bf16", "residual": "bf16", "group": 128},
        # a training step's norm of the widest model, residual stream kept in 32 bits
        {"name": "norm train", "op": "norm_train", "rows": 16384, "dim": 5120, "type": "bf16",
         "residual": "f32"},
        # odd rows and an odd width in 32 bits: no row but the first is aligned
        {"name": "norm train odd", "op": "norm_train", "rows": 4099, "dim": 1537, "type": "f32",
         "residual": "f32"},
        # one token for 128 sequences, state carried: latency
        {"name": "linrec step", "op": "linrec", "batch": 128, "seqlen": 1, "dim": 2560,
         "type": "bf16", "gate": True, "state": True, "packed": True},
        # the prefill of one long document: few channels, many steps
        {"name": "linrec long", "op": "linrec", "batch": 1, "seqlen": 65536, "dim": 1536,
         "type": "bf16", "gate": False, "state": False, "packed": False},
        # a training step on packed documents, f, x and z slices of one projection
        {"name": "linrec train", "op": "linrec_train", "batch": 8, "seqlen": 2048, "dim": 1536,
         "type": "bf16", "gate": True, "state": False, "packed": True},
        # odd sizes in 32 bits, resumed from a state
        {"name": "linrec train odd", "op": "linrec_train", "batch": 3, "seqlen": 1021,
         "dim": 777, "type": "f32", "gate": True, "state": True, "packed": False},
        # the loss of 8 tokens (one drafted continuation): bound by reading W once
        {"name": "ce few tokens", "op": "ce", "tokens": 8, "dim": 1536, "vocab": 50280},
        # evaluating a batch over a large vocabulary: the loss alone
        {"name": "ce evaluate", "op": "ce", "tokens": 4096, "dim": 1536, "vocab": 128000},
        # a small training batch
        {"name": "ce train", "op": "ce_train", "tokens": 2048, "dim": 1536, "vocab": 50280},
        # a full training batch over an odd vocabulary
        {"name": "ce train large", "op": "ce_train", "tokens": 8192, "dim": 2048,
         "vocab": 50257},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_q8", "norm_train", "linrec", "linrec_train", "ce",
                     "ce_train"])
    if op.startswith("norm"):
        rows, dim = _log_int(rng, 1, 32768), _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            dim = max(64, dim // 64 * 64)
        kind, res = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        case = {"op": op, "rows": rows, "dim": dim, "type": kind, "residual": res}
        if op == "norm_q8":
            case["group"] = rng.choice([0, 32, 128])
        return case
    if op.startswith("linrec"):
        seqlen, dim = _log_int(rng, 1, 65536), _log_int(rng, 16, 5120)
        if rng.random() < 0.6:
            dim = max(16, dim // 16 * 16)
        batch = _log_int(rng, 1, 256)
        most = 65536 * 1536 if op == "linrec" else 8 * 2048 * 2048
        batch = max(1, min(batch, most // (seqlen * dim)))
        seqlen = min(seqlen, most // dim)
        gate = rng.random() < 0.5
        return {"op": op, "batch": batch, "seqlen": seqlen, "dim": dim,
                "type": rng.choice(["bf16", "bf16", "f32"]), "gate": gate,
                "state": rng.random() < 0.5,
                # a slice of a packed projection starts on a 16-byte boundary
                "packed": gate and dim % 8 == 0 and rng.random() < 0.5}
    tokens = _log_int(rng, 1, 8192)
    dim = 8 * _log_int(rng, 16, 512)
    vocab = _log_int(rng, 1000, 128000)
    most = 8192 * 2048 * 50257
    tokens = max(1, min(tokens, most // (dim * vocab)))
    return {"op": op, "tokens": tokens, "dim": dim, "vocab": vocab}


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, e, r = case["rows"] * case["dim"], _SIZE[case["type"]], _SIZE[case["residual"]]
        fwd = n * (e + 2 * r) + 4 * case["dim"]           # x, residual and the sum, weight
        if op == "norm":
            return {"bytes": fwd + n * e, "flops": 6 * n}
        if op == "norm_q8":
            groups = 1 if case["group"] == 0 else -(-case["dim"] // case["group"])
            return {"bytes": fwd + n + 4 * case["rows"] * groups, "flops": 8 * n}
        # y, then dy, the sum's own gradient, the residual's gradient, dx where it has
        # another type, and the weight's gradient
        more = n * (2 * e + 2 * r + (e if e != r else 0)) + 4 * case["dim"]
        return {"bytes": fwd + more, "flops": 18 * n}
    if op.startswith("linrec"):
        b, d, e = case["batch"], case["dim"], _SIZE[case["type"]]
        n = b * case["seqlen"] * d
        streams = 4 if case["gate"] else 3                  # f, x, z and y
        states = (2 if case["state"] else 1) * 4 * b * d    # initial and final state
        if op == "linrec":
            return {"bytes": n * streams * e + states, "flops": 12 * n}
        # dy, df, dx and dz, the final state's gradient and the initial state's
        return {"bytes": 2 * n * streams * e + 2 * states, "flops": 40 * n}
    t, d, v = case["tokens"], case["dim"], case["vocab"]
    if op == "ce":
        return {"bytes": 2 * (t + v) * d + 16 * t, "flops": 2 * t * d * v}
    return {"bytes": 4 * (t + v) * d + 20 * t, "flops": 6 * t * d * v}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if op.startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        xt, rt = _TYPES[case["type"]], _TYPES[case["residual"]]
        s["x"] = randn(rows, dim).to(xt)
        s["residual"] = (3 * randn(rows, dim)).to(rt)
        s["weight"] = 1 + 0.1 * randn(dim)
        if op == "norm_train":
            s["dy"] = randn(rows, dim).to(xt)
            s["dsum"] = randn(rows, dim).to(rt)
        return s
    if op.startswith("linrec"):
        b, n, d, td = case["batch"], case["seqlen"], case["dim"], _TYPES[case["type"]]
        f = 2 + 1.5 * randn(b, n, d)
        if n > 64:
            # documents packed one after another: the gate's logit is -inf at a
            # document's first token, which starts its state anew
            starts = torch.rand(b, n, generator=g, device="cuda") < 1.0 / 512
            f = f.masked_fill(starts[..., None], float("-inf"))
        parts = [f, randn(b, n, d)] + ([randn(b, n, d)] if case["gate"] else [])
        if case["packed"]:
            parts = torch.cat(parts, -1).to(td).chunk(len(parts), -1)
        else:
            parts = [p.to(td) for p in parts]
        s["f"], s["x"] = parts[0], parts[1]
        s["z"] = parts[2] if case["gate"] else None
        s["h0"] = randn(b, d) if case["state"] else None
        if op == "linrec_train":
            s["dy"] = randn(b, n, d).to(td)
            s["dfinal"] = randn(b, d) if case["state"] else None
        return s
    t, d, v = case["tokens"], case["dim"], case["vocab"]
    s["h"] = randn(t, d).to(torch.bfloat16)
    s["W"] = (3 / math.sqrt(d) * randn(v, d)).to(torch.bfloat16)
    targets = torch.randint(0, v, (t,), generator=g, device="cuda")
    # padding and prompt tokens carry no loss
    skip = torch.rand(t, generator=g, device="cuda") < 0.03
    s["targets"] = targets.masked_fill(skip, -100)
    if op == "ce_train":
        # the gradient of the mean over the tokens that count
        s["dloss"] = torch.where(skip, 0.0, 1.0 / max(1, t - int(skip.sum())))
    return s


# -------------------------------------------------------------------- run

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import state_space_model_selective_gb300 as ssm

    op = s["case"]["op"]
    if op == "norm_q8":
        q, scales, total = ssm.ssm_add_rmsnorm_e4m3_fwd(s["x"], s["weight"], s["residual"],
                                                        eps=EPS, group=s["case"]["group"])
        return {"q": q, "scales": scales, "sum": total}
    if op.startswith("norm"):
        y, total = ssm.ssm_add_rmsnorm_fwd(s["x"], s["weight"], s["residual"], eps=EPS)
        if op == "norm":
            return {"y": y, "sum": total}
        g = ssm.ssm_add_rmsnorm_bwd(s["dy"], total, s["weight"], dsum=s["dsum"], eps=EPS)
        return {"y": y, "sum": total, "dx": g["dx"], "dresidual": g["dresidual"],
                "dweight": g["dweight"]}
    if op == "linrec":
        y, final = ssm.ssm_linrec_fwd(s["f"], s["x"], s["z"], initial_state=s["h0"])
        return {"y": y, "final": final}
    if op == "linrec_train":
        b, n, d = s["x"].shape
        kept = torch.empty(ssm.ssm_linrec_checkpoint_bytes(b, n, d) // 4, device=s["x"].device)
        y, final = ssm.ssm_linrec_fwd(s["f"], s["x"], s["z"], initial_state=s["h0"],
                                      checkpoints=kept)
        g = ssm.ssm_linrec_bwd(s["f"], s["x"], s["dy"], s["z"], initial_state=s["h0"],
                               dfinal_state=s["dfinal"], checkpoints=kept,
                               want_dinitial_state=s["h0"] is not None)
        return {"y": y, "final": final, "df": g["df"], "dx": g["dx"], "dz": g["dz"],
                "dh0": g["dinitial_state"]}
    loss, lse = ssm.ssm_vocab_ce_fwd(s["h"], s["W"], s["targets"])
    if op == "ce":
        return {"loss": loss, "lse": lse}
    g = ssm.ssm_vocab_ce_bwd(s["h"], s["W"], s["targets"], lse, s["dloss"])
    return {"loss": loss, "lse": lse, "dh": g["dh"], "dW": g["dW"]}


def _plain(s):
    op = s["case"]["op"]
    if op.startswith("norm"):
        return _plain_norm(s)
    if op.startswith("linrec"):
        return _plain_linrec(s)
    return _plain_ce(s)


def _plain_norm(s):
    op, xt, rt = s["case"]["op"], s["x"].dtype, s["residual"].dtype
    total = s["x"].float() + s["residual"].float()
    r = torch.rsqrt((total * total).mean(-1, keepdim=True) + EPS)
    y = total * r * s["weight"]
    kept = total.to(rt)
    if op == "norm":
        return {"y": y.to(xt), "sum": kept}
    if op == "norm_q8":
        rows, dim = y.shape
        group = s["case"]["group"] or dim
        pad = -dim % group
        yg = torch.cat([y, y.new_zeros(rows, pad)], -1) if pad else y
        yg = yg.reshape(rows, -1, group)
        amax = yg.abs().amax(-1, keepdim=True)
        q = torch.where(amax > 0, yg * (E4M3_MAX / amax), 0.0).clamp(-E4M3_MAX, E4M3_MAX)
        q = q.reshape(rows, -1)[:, :dim].contiguous().to(torch.float8_e4m3fn)
        return {"q": q, "scales": (amax / E4M3_MAX).squeeze(-1), "sum": kept}
    # the gradient is taken at the sum as it was kept
    t = kept.float()
    r = torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)
    n, dy = t * r, s["dy"].float()
    gw = dy * s["weight"]
    d = r * (gw - n * (gw * n).mean(-1, keepdim=True)) + s["dsum"].float()
    return {"y": y.to(xt), "sum": kept, "dx": d.to(xt), "dresidual": d.to(rt),
            "dweight": (dy * n).sum(0)}


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 from h_{-1} = 0, by doubling: after the
    step of width k, (a, b) at t stand for the 2 k steps that end there."""
    k, n = 1, a.shape[1]
    while k < n:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _plain_linrec(s):
    td, h0 = s["x"].dtype, s["h0"]
    f, x = s["f"].float(), s["x"].float()
    a, om = 1 / (1 + torch.exp(-f)), 1 / (1 + torch.exp(f))
    b = om * x
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    h = _scan(a, b)
    out = {"final": h[:, -1].contiguous()}
    if s["z"] is not None:
        z = s["z"].float()
        sg = 1 / (1 + torch.exp(-z))
        out["y"] = (h * z * sg).to(td)
    else:
        out["y"] = h.to(td)
    if s["case"]["op"] == "linrec":
        return out
    dy = s["dy"].float()
    dh = dy if s["z"] is None else dy * z * sg
    if s["dfinal"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dfinal"][:, None]], 1)
    # the adjoint runs backwards in time: lam_t = dh_t + a_{t+1} lam_{t+1}
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    lam = _scan(nxt.flip(1), dh.flip(1)).flip(1)
    first = torch.zeros_like(h[:, 0]) if h0 is None else h0
    prev = torch.cat([first[:, None], h[:, :-1]], 1)
    out["df"] = (lam * (prev - x) * a * om).to(td)
    out["dx"] = (lam * om).to(td)
    out["dz"] = None if s["z"] is None else (dy * h * sg * (1 + z * (1 - sg))).to(td)
    out["dh0"] = None if h0 is None else a[:, 0] * lam[:, 0]
    return out


def _plain_ce(s):
    h, w, targets = s["h"].float(), s["W"].float(), s["targets"]
    logits = h @ w.t()
    m = logits.amax(-1, keepdim=True)
    lse = (m + torch.log(torch.exp(logits - m).sum(-1, keepdim=True))).squeeze(-1)
    counts = targets >= 0
    at = targets.clamp(min=0)[:, None]
    loss = torch.where(counts, lse - logits.gather(1, at).squeeze(-1), 0.0)
    if s["case"]["op"] == "ce":
        return {"loss": loss, "lse": lse}
    p = torch.exp(logits - lse[:, None])
    p.scatter_add_(1, at, -torch.ones_like(at, dtype=p.dtype))
    p *= torch.where(counts, s["dloss"], 0.0)[:, None]
    return {"loss": loss, "lse": lse, "dh": (p @ w).to(torch.bfloat16),
            "dW": (p.t() @ h).to(torch.bfloat16)}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definition in 64 bits: the recurrence step by step, the softmax with its
    full matrix of logits, the norm's gradient from the quotient's derivative."""
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(s)
    if op.startswith("linrec"):
        return _exact_linrec(s)
    return _exact_ce(s)


def _exact_norm(s):
    case = s["case"]
    dim = case["dim"]
    total = s["x"].double() + s["residual"].double()
    y = total / (total.square().sum(-1, keepdim=True) / dim + EPS).sqrt() * s["weight"].double()
    if case["op"] == "norm":
        return {"y": y, "sum": total}
    if case["op"] == "norm_q8":
        parts, scales = [], []
        for c0 in range(0, dim, case["group"] or dim):
            piece = y[:, c0:c0 + (case["group"] or dim)]
            scale = piece.abs().max(-1, keepdim=True).values / E4M3_MAX
            parts.append((piece / scale).to(torch.float8_e4m3fn).double())
            scales.append(scale)
        return {"q": torch.cat(parts, -1), "scales": torch.cat(scales, -1), "sum": total}
    t = total.to(s["residual"].dtype).double()
    rms = (t.square().sum(-1, keepdim=True) / dim + EPS).sqrt()
    dn = s["dy"].double() * s["weight"].double()
    d = dn / rms - t * (dn * t).sum(-1, keepdim=True) / (dim * rms ** 3) + s["dsum"].double()
    return {"y": y, "sum": total, "dx": d, "dresidual": d,
            "dweight": (s["dy"].double() * t / rms).sum(0)}


def _exact_linrec(s):
    f, x = s["f"].double(), s["x"].double()
    b, n, d = x.shape
    a, om = torch.sigmoid(f), torch.sigmoid(-f)
    h = torch.zeros(b, d, dtype=torch.float64, device=x.device)
    if s["h0"] is not None:
        h = s["h0"].double()
    first, hs = h, torch.empty_like(x)
    for t in range(n):
        h = a[:, t] * h + om[:, t] * x[:, t]
        hs[:, t] = h
    z = s["z"].double() if s["z"] is not None else None
    gate = z * torch.sigmoid(z) if z is not None else torch.ones_like(hs)
    out = {"y": hs * gate, "final": h}
    if s["case"]["op"] == "linrec":
        return out
    dy = s["dy"].double()
    lam = torch.zeros_like(first)
    if s["dfinal"] is not None:
        lam = s["dfinal"].double()
    df, dx = torch.empty_like(x), torch.empty_like(x)
    for t in range(n - 1, -1, -1):
        lam = lam + dy[:, t] * gate[:, t]
        before = hs[:, t - 1] if t else first
        df[:, t] = lam * (before - x[:, t]) * a[:, t] * om[:, t]
        dx[:, t] = lam * om[:, t]
        lam = a[:, t] * lam
    out.update(df=df, dx=dx, dz=None, dh0=lam if s["h0"] is not None else None)
    if z is not None:
        sg = torch.sigmoid(z)
        out["dz"] = dy * hs * (sg + z * sg * (1 - sg))
    return out


def _exact_ce(s):
    h, w, targets = s["h"].double(), s["W"].double(), s["targets"]
    logits = torch.matmul(h, w.transpose(0, 1))
    lse = torch.logsumexp(logits, -1)
    rows = torch.nonzero(targets >= 0).squeeze(-1)
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - logits[rows, targets[rows]]
    if s["case"]["op"] == "ce":
        return {"loss": loss, "lse": lse}
    p = torch.softmax(logits, -1)
    p[rows, targets[rows]] -= 1
    skipped = torch.ones_like(lse).index_fill_(0, rows, 0.0).bool()
    p = torch.where(skipped[:, None], 0.0, p) * s["dloss"].double()[:, None]
    return {"loss": loss, "lse": lse, "dh": torch.matmul(p, w),
            "dW": torch.matmul(p.transpose(0, 1), h)}
