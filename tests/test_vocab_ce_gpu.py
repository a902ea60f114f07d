"""Softmax cross entropy over a vocabulary (ssm_vocab_ce_fwd, ssm_vocab_ce_bwd)
against the plain 64-bit form on the same inputs.

Tolerances, derived.  Logits are exact bf16 products summed in fp32: with K terms
of size up to l the rounding stays below about sqrt(K) 2^-24 l, 3e-6 l here, and
exp, log and the sums over columns add a few roundings, so loss and lse are
within 1e-5 of max(1, |lse|).  P is rounded to bf16, at most 2^-9 of each value,
independently: a sum of n such products is off by 2^-9 times the root of the
sum of their squares, which is taken from the 64-bit P; six of those, plus 1e-5 of
the largest value for the fp32 sums, plus 2^-8 of the value for a bf16 result."""
import numpy as np
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests import plain64 as P
from tests.helpers import to64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _inputs(tokens, dim, vocab, seed, skip=0.1):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(tokens, dim, generator=g).to(BF16)
    W = (3 / dim ** 0.5 * torch.randn(vocab, dim, generator=g)).to(BF16)
    t = torch.randint(0, vocab, (tokens,), generator=g)
    t[torch.rand(tokens, generator=g) < skip] = -100
    return h, W, t, torch.rand(tokens, generator=g) + 0.1


def _check_loss(got, ref, lse):
    got = to64(got)
    assert np.all(np.isfinite(got))
    assert np.max(np.abs(got - ref) / np.maximum(1.0, np.abs(lse))) <= 1e-5


def _check_grads(g, h, W, t, d, dtype):
    h64, W64, t64, d64 = to64(h), to64(W), t.numpy(), to64(d)
    dh, dW = P.ce_bwd(h64, W64, t64, d64)
    p = np.exp(h64 @ W64.T - P.ce_fwd(h64, W64, t64)[1][:, None])
    rows = np.flatnonzero(t64 >= 0)
    p[rows, t64[rows]] -= 1
    p *= np.where(t64 >= 0, d64, 0.0)[:, None]
    for name, ref, spread in (("dh", dh, np.sqrt((p * p) @ (W64 * W64))),
                              ("dW", dW, np.sqrt((p * p).T @ (h64 * h64)))):
        got = to64(g[name])
        assert got.shape == ref.shape and g[name].dtype == dtype
        assert np.all(np.isfinite(got)), name
        lim = 6 * 2.0 ** -9 * spread + 1e-5 * np.max(np.abs(ref))
        if dtype == BF16:
            lim = lim + 2.0 ** -8 * np.abs(ref)
        over = np.abs(got - ref) - lim
        assert np.max(over) <= 0, (name, float(np.max(over)), int((over > 0).sum()))


# one token; rows and columns short of, at and past a tile's 128 and 256; widths
# below one stage's 64, off its multiple and past several rounds of the ring;
# vocabularies of one value and off every multiple
SIZES = [(1, 8, 1), (1, 64, 7), (3, 72, 300), (127, 128, 129), (128, 64, 256), (129, 200, 257),
         (256, 1024, 512), (257, 1544, 1001), (300, 40, 5000), (1000, 264, 2049), (5, 2048, 20011),
         (600, 512, 9000)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_matches_plain(size, dtype):
    h, W, t, d = _inputs(*size, sum(size))
    hc, Wc, tc, dc = h.cuda(), W.cuda(), t.cuda(), d.cuda()
    loss, lse = binding.ssm_vocab_ce_fwd(hc, Wc, tc)
    loss_ref, lse_ref = P.ce_fwd(to64(h), to64(W), t.numpy())
    _check_loss(lse, lse_ref, lse_ref)
    _check_loss(loss, loss_ref, lse_ref)
    g = binding.ssm_vocab_ce_bwd(hc, Wc, tc, lse, dc, grad_dtype=dtype)
    _check_grads(g, h, W, t, d, dtype)


def test_several_pieces(monkeypatch):
    """More tokens than a piece of the whole vocabulary fits: two pieces, the second
    narrower and ending inside a tile."""
    tokens, dim, vocab = 20000, 64, 7001
    h, W, t, d = _inputs(tokens, dim, vocab, 5)
    need = binding.ssm_vocab_ce_bwd_workspace_bytes(tokens, dim, vocab)
    assert need < tokens * vocab * 2, need  # not the whole P
    hc, Wc, tc, dc = h.cuda(), W.cuda(), t.cuda(), d.cuda()
    _, lse = binding.ssm_vocab_ce_fwd(hc, Wc, tc)
    g = binding.ssm_vocab_ce_bwd(hc, Wc, tc, lse, dc, grad_dtype=F32)
    _check_grads(g, h, W, t, d, F32)


@pytest.mark.parametrize("tokens", [5, 200])
def test_targets_without_loss(tokens):
    """Negative targets of any value carry nothing; with none that counts every
    gradient is exactly 0.  A target past the vocabulary gives a NaN loss and no
    gradient."""
    h, W, t, d = _inputs(tokens, 72, 300, 6, skip=0)
    t[0], t[1], t[2] = -1, torch.iinfo(torch.int64).min, 300
    loss, lse = binding.ssm_vocab_ce_fwd(h.cuda(), W.cuda(), t.cuda())
    assert not loss[:2].any() and loss[2].isnan() and loss[3:].isfinite().all()
    assert lse.isfinite().all()
    g = binding.ssm_vocab_ce_bwd(h.cuda(), W.cuda(), t.cuda(), lse, d.cuda(), grad_dtype=F32)
    t[2] = -1
    _check_grads(g, h, W, t, d, F32)
    none = torch.full_like(t, -100).cuda()
    g = binding.ssm_vocab_ce_bwd(h.cuda(), W.cuda(), none, lse, d.cuda(), grad_dtype=F32)
    assert not g["dh"].any() and not g["dW"].any()


def test_large_and_equal_logits():
    """Logits of hundreds (the maximum keeps exp in range), and a row whose logits
    are all equal: lse = log(vocab) + l."""
    h, W, t, d = _inputs(130, 64, 1000, 7, skip=0)
    h[:64] *= 100
    h[64:70] = 0
    loss, lse = binding.ssm_vocab_ce_fwd(h.cuda(), W.cuda(), t.cuda())
    loss_ref, lse_ref = P.ce_fwd(to64(h), to64(W), t.numpy())
    _check_loss(lse, lse_ref, lse_ref)
    _check_loss(loss, loss_ref, lse_ref)
    np.testing.assert_allclose(to64(lse[64:70]), np.log(1000.0), rtol=1e-6)
    # gradient of confident rows: P near 0 but for a few columns
    g = binding.ssm_vocab_ce_bwd(h[64:].contiguous().cuda(), W.cuda(), t[64:].contiguous().cuda(),
                                 lse[64:].contiguous(), d[64:].contiguous().cuda(), grad_dtype=F32)
    _check_grads(g, h[64:], W, t[64:], d[64:], F32)


def test_nan_stays_in_its_token():
    h, W, t, _ = _inputs(40, 64, 500, 8, skip=0)
    h[7, 3] = float("nan")
    loss, lse = binding.ssm_vocab_ce_fwd(h.cuda(), W.cuda(), t.cuda())
    assert loss[7].isnan() and lse[7].isnan()
    rest = [i for i in range(40) if i != 7]
    loss_ref, lse_ref = P.ce_fwd(to64(h)[rest], to64(W), t.numpy()[rest])
    _check_loss(lse[rest], lse_ref, lse_ref)
    _check_loss(loss[rest], loss_ref, lse_ref)


def test_no_tokens():
    _, W, _, _ = _inputs(1, 64, 500, 9)
    h, t = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, dtype=torch.int64,
                                                                      device="cuda")
    e = torch.empty(0, device="cuda")
    loss, lse = binding.ssm_vocab_ce_fwd(h, W.cuda(), t)
    assert loss.shape == (0,) and lse.shape == (0,)
    g = binding.ssm_vocab_ce_bwd(h, W.cuda(), t, e, e)
    assert g["dh"].shape == (0, 64) and not g["dW"].any()


def test_bit_equal_and_another_stream():
    h, W, t, d = (v.cuda() for v in _inputs(700, 320, 3001, 10))
    loss, lse = binding.ssm_vocab_ce_fwd(h, W, t)
    g = binding.ssm_vocab_ce_bwd(h, W, t, lse, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    for _ in range(3):
        a, b = binding.ssm_vocab_ce_fwd(h, W, t, stream=side)
        runs.append((a, b, binding.ssm_vocab_ce_bwd(h, W, t, b, d, stream=side)))
    torch.cuda.synchronize()
    for a, b, r in runs:
        assert torch.equal(a, loss) and torch.equal(b, lse)
        assert torch.equal(r["dh"], g["dh"]) and torch.equal(r["dW"], g["dW"])


def test_writes_stay_inside_the_outputs():
    h, W, t, d = (v.cuda() for v in _inputs(131, 72, 301, 11))
    before = [v.clone() for v in (h, W, t, d)]

    def guarded(shape, dt):
        num = int(np.prod(shape))
        buf = torch.full((num + 128,), -7.25e33, dtype=dt, device="cuda")
        buf[64:64 + num] = float("nan")
        return buf, buf[64:64 + num].view(shape)

    for dt in (BF16, F32):
        ws = [torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda") for n in
              (binding.ssm_vocab_ce_workspace_bytes(131, 72, 301),
               binding.ssm_vocab_ce_bwd_workspace_bytes(131, 72, 301))]
        bufs = {"loss": guarded((131,), F32), "lse": guarded((131,), F32),
                "dh": guarded((131, 72), dt), "dW": guarded((301, 72), dt)}
        binding.ssm_vocab_ce_fwd(h, W, t, loss=bufs["loss"][1], lse=bufs["lse"][1],
                                 workspace=ws[0][:-256])
        binding.ssm_vocab_ce_bwd(h, W, t, bufs["lse"][1], d, grad_dtype=dt, workspace=ws[1][:-256],
                                 out={"dh": bufs["dh"][1], "dW": bufs["dW"][1]})
        torch.cuda.synchronize()
        for w in ws:
            assert (w[-256:] == 77).all()
            assert binding.ssm_last_device_status(w) == 0
        for k, (buf, v) in bufs.items():
            guard = torch.full((64,), -7.25e33, dtype=buf.dtype, device="cuda")
            assert torch.equal(buf[:64], guard) and torch.equal(buf[-64:], guard), k
            assert not v.isnan().any(), k
    for v, b in zip((h, W, t, d), before):
        assert torch.equal(v, b)


# few tokens: the columns of the vocabulary-major kernel (16, 32 or 64, full and not)
# and the first size past it; vocabularies cut among the CTAs into whole tiles, part
# of a tile, part of a box of 16 rows, and into fewer pieces than there are CTAs
@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("dim,vocab", [(64, 15), (520, 2433), (72, 20011), (136, 60000)])
def test_few_tokens(tokens, dim, vocab):
    h, W, t, d = _inputs(tokens, dim, vocab, tokens + vocab)
    loss, lse = binding.ssm_vocab_ce_fwd(h.cuda(), W.cuda(), t.cuda())
    loss_ref, lse_ref = P.ce_fwd(to64(h), to64(W), t.numpy())
    _check_loss(lse, lse_ref, lse_ref)
    _check_loss(loss, loss_ref, lse_ref)


@pytest.mark.parametrize("tokens", [9, 131])
def test_vectors_off_a_16_byte_boundary(tokens):
    """Targets, lse and dloss as ranges that start at the second element (a program's labels
    shifted by one): the same results, on the current stream and on another."""
    h, W, t, d = (v.cuda() for v in _inputs(tokens, 72, 300, 12))
    loss, lse = binding.ssm_vocab_ce_fwd(h, W, t)
    g = binding.ssm_vocab_ce_bwd(h, W, t, lse, d)
    shifted = [torch.cat([v.new_zeros(1), v])[1:] for v in (t, lse, d)]
    assert all(v.data_ptr() % 16 and v.is_contiguous() for v in shifted)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        a, b = binding.ssm_vocab_ce_fwd(h, W, shifted[0], stream=stream)
        r = binding.ssm_vocab_ce_bwd(h, W, *shifted, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(a, loss) and torch.equal(b, lse)
        assert torch.equal(r["dh"], g["dh"]) and torch.equal(r["dW"], g["dW"])


@pytest.mark.parametrize("tokens", [1, 6, 15, 16, 17, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("dim,vocab", [(64, 15), (520, 2433), (72, 20011), (136, 60000)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_few_tokens_gradient(tokens, dim, vocab, dtype):
    """The gradient's own kernel of few tokens, in each of its widths, full and not, and the
    first size past it; every fourth target lies outside the vocabulary, on either side."""
    h, W, t, d = _inputs(tokens, dim, vocab, tokens + vocab, skip=0)
    counts = torch.arange(tokens) % 4 != 2
    t[~counts] = torch.where(torch.arange(tokens) % 8 == 2, -1, vocab)[~counts]
    hc, Wc, tc, dc = h.cuda(), W.cuda(), t.cuda(), d.cuda()
    _, lse = binding.ssm_vocab_ce_fwd(hc, Wc, tc)
    g = binding.ssm_vocab_ce_bwd(hc, Wc, tc, lse, dc, grad_dtype=dtype)
    assert not g["dh"][~counts.cuda()].any()
    t[~counts] = -1
    _check_grads(g, h, W, t, d, dtype)
