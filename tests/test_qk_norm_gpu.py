"""Norms of query and key heads with the rotation by position (ssm_qk_norm_rope_fwd,
_bwd) against the plain 64-bit form on the same inputs.

Tolerances, derived, as parts of the head's largest value: a sum of up to 256 squares
(lanes of 16 in a row, then 4 shuffles: at most 20 roundings of 2^-24, halved by the
root), the root's 2 ulp, the products with it and the weight, a sine and cosine off by
2 ulp and two more roundings: below 2e-6 forward, 4e-6 in the gradient, where a second sum
of that kind enters.  A bf16 value adds half a step, 2^-8 of itself.  dw is a sum over
tokens and heads of terms of either sign, off by about sqrt(terms) roundings of its
largest partial sums: 1e-5 of its largest value."""
import numpy as np
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests import plain64_heads as H
from tests.helpers import to64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


def near(got, ref, dtype, what, tol):
    got = to64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    scale = np.max(np.abs(ref), axis=-1, keepdims=True)
    lim = tol * scale + (2.0 ** -8 * np.abs(ref) * (1 + 1e-3) if dtype == BF16 else 0.0)
    over = np.abs(got - ref) - lim
    assert np.all(over <= 0), (what, float(over.max()))


def inputs(b, n, hq, hk, d, rot, xt, seed, far=0):
    g = torch.Generator().manual_seed(seed)
    q = (2 * torch.randn(b, n, hq, d, generator=g)).to(xt)
    k = (0.3 * torch.randn(b, n, hk, d, generator=g)).to(xt)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    pos = far + torch.randint(0, 5000, (b, n), generator=g)
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else None
    return q, k, wq, wk, pos, freq


def check(q, k, wq, wk, pos, freq, inter, yt, seed=0, put=lambda t: t.cuda()):
    xt, rot = q.dtype, 0 if freq is None else 2 * len(freq)
    cuda = [None if t is None else t.cuda() for t in (wq, wk, pos, freq)]
    args = dict(zip(("q_weight", "k_weight", "positions", "inv_freq"), cuda), eps=EPS,
                interleaved=inter)
    qd, kd = put(q), None if k is None else put(k)
    phase = H.angles(to64(pos), to64(freq)) if rot else None
    outs = binding.ssm_qk_norm_rope_fwd(qd, kd, out_dtype=yt, **args)
    g = torch.Generator().manual_seed(seed + 1)
    dys = [None if x is None else torch.randn(x.shape, generator=g).to(yt) for x in (q, k)]
    grads = binding.ssm_qk_norm_rope_bwd(*(None if t is None else t.cuda() for t in dys), qd, kd,
                                         **args)
    for x, w, y, dy, name in ((q, wq, outs[0], dys[0], "q"), (k, wk, outs[1], dys[1], "k")):
        if x is None:
            assert y is None and grads["dk"] is None and grads["dk_weight"] is None
            continue
        w = None if w is None else to64(w)
        near(y, H.qk_fwd(to64(x), w, phase, rot, EPS, inter), yt, name, 2e-6)
        dx, dw = H.qk_bwd(to64(x), w, phase, rot, EPS, to64(dy), inter)
        near(grads["d" + name], dx, xt, "d" + name, 4e-6)
        assert y.dtype == yt and grads["d" + name].dtype == xt
        if w is None:
            assert grads[f"d{name}_weight"] is None
        else:
            near(grads[f"d{name}_weight"], dw, F32, f"d{name}_weight", 1e-5)
    return outs, grads


# rot as columns: none, two, halves that are and are not multiples of 8, all of them
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dim,rot", [(8, 0), (8, 2), (8, 8), (16, 16), (24, 12), (64, 64),
                                     (72, 20), (72, 32), (128, 128), (128, 64), (136, 136),
                                     (200, 16), (248, 246), (256, 256), (256, 128)])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)],
                         ids=lambda t: "-".join(str(v)[6:] for v in t))
def test_forward_and_gradient(dim, rot, inter, types):
    check(*inputs(2, 19, 5, 3, dim, rot, types[0], dim + rot), inter, types[1])


@pytest.mark.parametrize("b,n,hq,hk", [(1, 1, 1, 1), (1, 1, 32, 8), (3, 1, 7, 2), (1, 700, 2, 1),
                                       (2, 333, 33, 5), (1, 5000, 1, 1), (5, 3, 130, 1)])
def test_counts_of_tokens_and_heads(b, n, hq, hk):
    check(*inputs(b, n, hq, hk, 64, 64, BF16, n), False, BF16)
    check(*inputs(b, n, hq, hk, 40, 12, F32, n), False, F32)


def test_queries_alone_and_no_weights():
    q, k, wq, wk, pos, freq = inputs(2, 9, 3, 2, 32, 32, F32, 5)
    check(q, None, wq, None, pos, freq, False, F32)
    check(q, k, None, wk, pos, freq, True, F32)
    check(q, k, None, None, pos, None, False, F32)


def test_empty():
    q, k, wq, wk, pos, freq = inputs(2, 0, 3, 2, 32, 32, F32, 5)
    args = dict(q_weight=wq.cuda(), k_weight=wk.cuda(), positions=pos.cuda(), inv_freq=freq.cuda())
    outs = binding.ssm_qk_norm_rope_fwd(q.cuda(), k.cuda(), **args)
    assert outs[0].shape == q.shape and outs[1].shape == k.shape
    g = binding.ssm_qk_norm_rope_bwd(q.cuda(), k.cuda(), q.cuda(), k.cuda(), **args)
    assert not g["dq_weight"].any() and not g["dk_weight"].any()


@pytest.mark.parametrize("far", [1 << 20, 1 << 33, -(1 << 20)])
def test_far_positions(far):
    """The phase is exact modulo a turn at any position: at 2^33 it is off by up to 2^-52 *
    2^33 / (2 pi) turns, 5e-7 rad, inside the tolerance at the weights' size."""
    check(*inputs(2, 17, 3, 2, 64, 64, F32, 7, far=far), False, F32)


@pytest.mark.parametrize("xt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 8, 1, 3])
def test_ranges_of_a_projection(xt, shift):
    """q and k as column ranges of one projection, aligned to 16 bytes and not."""
    q, k, wq, wk, pos, freq = inputs(3, 11, 4, 2, 48, 48, xt, shift)
    b, n = q.shape[:2]
    whole = torch.randn(b, n, 6 * 48 + 9 + shift, dtype=torch.float32).to(xt)
    whole[..., shift:shift + 192], whole[..., shift + 192:shift + 288] = q.flatten(2), k.flatten(2)
    whole = whole.cuda()
    parts = {4: whole[..., shift:shift + 192].unflatten(-1, (4, 48)),
             2: whole[..., shift + 192:shift + 288].unflatten(-1, (2, 48))}
    kept = whole.clone()
    check(q, k, wq, wk, pos, freq, False, xt, put=lambda t: parts[t.shape[2]])
    assert torch.equal(whole, kept)


def test_zero_heads_and_nan_stay_in_their_rows():
    q, k, wq, wk, pos, freq = inputs(1, 40, 4, 4, 64, 64, F32, 9)
    q[0, 3, 1] = 0
    args = dict(q_weight=wq.cuda(), k_weight=wk.cuda(), positions=pos.cuda(),
                inv_freq=freq.cuda(), eps=EPS)
    clean = binding.ssm_qk_norm_rope_fwd(q.cuda(), k.cuda(), **args)
    assert not clean[0][0, 3, 1].any()
    q[0, 5, 2, 7] = float("nan")
    k[0, 6, 0, 0] = float("inf")
    outs = binding.ssm_qk_norm_rope_fwd(q.cuda(), k.cuda(), **args)
    bad_q, bad_k = torch.zeros(1, 40, 4, dtype=torch.bool), torch.zeros(1, 40, 4, dtype=torch.bool)
    bad_q[0, 5, 2] = bad_k[0, 6, 0] = True
    assert outs[0].cpu()[bad_q].isnan().all() and outs[1].cpu()[bad_k].isnan().any()
    assert torch.equal(outs[0].cpu()[~bad_q], clean[0].cpu()[~bad_q])
    assert torch.equal(outs[1].cpu()[~bad_k], clean[1].cpu()[~bad_k])


def test_runs_are_bit_equal_on_another_stream_and_in_a_graph():
    q, k, wq, wk, pos, freq = (t.cuda() for t in inputs(2, 300, 8, 4, 128, 128, BF16, 3))
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    args = dict(q_weight=wq, k_weight=wk, positions=pos, inv_freq=freq, eps=EPS)

    def both(stream=None):
        outs = binding.ssm_qk_norm_rope_fwd(q, k, stream=stream, **args)
        return list(outs) + list(binding.ssm_qk_norm_rope_bwd(dq, dk, q, k, stream=stream,
                                                              **args).values())

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, kept):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_guards_around_the_outputs():
    """Nothing is written outside the outputs (odd sizes, several tiles)."""
    q, k, wq, wk, pos, freq = (t.cuda() for t in inputs(1, 77, 3, 2, 72, 20, BF16, 4))
    shapes = {"q_out": q.shape, "k_out": k.shape, "dq": q.shape, "dk": k.shape,
              "dq_weight": (72,), "dk_weight": (72,)}
    bufs, views = {}, {}
    for name, shape in shapes.items():
        dt = F32 if "weight" in name else BF16
        size = int(np.prod(shape))
        bufs[name] = torch.full((size + 128,), 7.0, dtype=dt, device="cuda")
        views[name] = bufs[name][64:64 + size].view(shape)
    args = dict(q_weight=wq, k_weight=wk, positions=pos, inv_freq=freq, eps=EPS)
    binding.ssm_qk_norm_rope_fwd(q, k, q_out=views["q_out"], k_out=views["k_out"], **args)
    binding.ssm_qk_norm_rope_bwd(q, k, q, k, out={n: views[n] for n in
                                                  ("dq", "dk", "dq_weight", "dk_weight")}, **args)
    for name, b in bufs.items():
        assert torch.all(b[:64] == 7) and torch.all(b[-64:] == 7), name


def test_a_tile_of_tokens_far_apart():
    """Rows of a wide projection: a tile is shortened so that its bytes count in 31 bits."""
    wide = torch.zeros(1, 40, 1 << 24, dtype=BF16, device="cuda")
    q, _, wq, _, pos, freq = inputs(1, 40, 2, 1, 64, 64, BF16, 6)
    wide[..., 1 << 20:(1 << 20) + 128] = q.flatten(2).cuda()
    part = wide[..., 1 << 20:(1 << 20) + 128].unflatten(-1, (2, 64))
    args = dict(q_weight=wq.cuda(), positions=pos.cuda(), inv_freq=freq.cuda())
    near_, _ = binding.ssm_qk_norm_rope_fwd(q.cuda(), **args)
    far_, _ = binding.ssm_qk_norm_rope_fwd(part, **args)
    assert torch.equal(near_, far_)


@pytest.mark.parametrize("n,hq,hk,d,rot", [(4099, 32, 8, 128, 64), (5003, 5, 3, 128, 128), (8133, 4, 1, 64, 0),
                                           (8133, 7, 0, 64, 48), (4003, 1, 4, 256, 256), (30001, 3, 1, 16, 16),
                                           (30001, 3, 2, 32, 16), (4099, 4, 12, 128, 128), (4097, 0, 8, 128, 32),
                                           (5003, 8, 16, 64, 64), (4003, 6, 2, 256, 128), (3700, 64, 32, 16, 16)])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, F32), (BF16, F32)])
def test_many_tokens(n, hq, hk, d, rot, xt, yt):
    """Enough tokens for whole tiles in all CTAs: lanes hold their angles over the heads."""
    q, k, wq, wk, pos, freq = inputs(1, n, hq, max(hk, 1), d, rot, xt, n + d)
    check(q, k if hk else None, wq, wk if hk else None, pos, freq, False, yt)
    if (xt, yt) == (BF16, BF16) and hk and hq:  # ranges of a projection give the same, bit for bit
        wide = torch.cat((q.flatten(2), k.flatten(2)), -1).cuda()
        qr = wide[..., :hq * d].unflatten(-1, (hq, d))
        kr = wide[..., hq * d:].unflatten(-1, (hk, d))
        args = dict(q_weight=wq.cuda(), positions=pos.cuda(), inv_freq=None if freq is None else freq.cuda())
        for a, b in zip(binding.ssm_qk_norm_rope_fwd(q.cuda(), k.cuda(), **args),
                        binding.ssm_qk_norm_rope_fwd(qr, kr, **args)):
            assert torch.equal(a, b)
