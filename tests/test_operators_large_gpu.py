"""Tensors of more than 2^31 elements through the norm, the recurrence and the cross
entropy: what lies at their ends is compared with the plain form, on the GPU in 64 bits.
Tolerances as in the operators' own tests."""
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests import plain64 as P
from tests.helpers import to64
from tests.test_linrec_gpu import _near as near_linrec
from tests.test_norm_gpu import _near as near_norm

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _randn(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape, dtype=BF16: torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


@pytest.mark.parametrize("dim", [8192, 1001])
def test_norm(dim):
    rows = (2 ** 31 + 2 ** 27) // dim
    randn = _randn(1)
    x, res, w = randn(rows, dim), randn(rows, dim), randn(dim, dtype=F32)
    y, s = binding.ssm_add_rmsnorm_fwd(x, w, res, eps=EPS)
    q, scales, _ = binding.ssm_add_rmsnorm_e4m3_fwd(x, w, res, eps=EPS, return_sum=False)
    g = binding.ssm_add_rmsnorm_bwd(x, s, w, eps=EPS)
    edge = 2 ** 31 // dim
    for at in (slice(0, 30), slice(edge - 15, edge + 15), slice(rows - 30, rows)):
        y_ref, s_ref = P.norm_fwd(to64(x[at]), to64(res[at]), to64(w), EPS)
        near_norm(y[at], y_ref, BF16, "y")
        near_norm(s[at], s_ref, BF16, "sum", 1e-6)
        amax = P.group_amax(y_ref, 128)
        near_norm(scales[at], amax / 448, F32, "scales")
        back = q[at].float().cpu().numpy() * scales[at].cpu().numpy().repeat(128, 1)[:, :dim]
        assert abs(back - y_ref).max() <= abs(y_ref).max() / 14  # half of a step of 3 bits
        dx_ref, _ = P.norm_bwd(to64(s[at]), to64(w), EPS, to64(x[at]))
        near_norm(g["dx"][at], dx_ref, BF16, "dx")
    dw = torch.zeros(dim, dtype=torch.float64, device="cuda")
    for r in range(0, rows, 16384):
        t = s[r:r + 16384].double()
        t *= torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)
        dw += (x[r:r + 16384].double() * t).sum(0)
    near_norm(g["dweight"], to64(dw), F32, "dweight", 1e-5)


@pytest.mark.parametrize("dim", [2048, 2047])
def test_linrec(dim):
    """The gates forget within some hundred steps, so that the last steps and the first ones
    are those of a short sequence."""
    n, m = (2 ** 31 + 2 ** 27) // dim, 600
    randn = _randn(2)
    f = randn(1, n, dim).mul_(0.5).add_(1)
    x, dy = randn(1, n, dim), randn(1, n, dim)
    kept = torch.empty(binding.ssm_linrec_checkpoint_bytes(1, n, dim) // 4, device="cuda")
    y, fin = binding.ssm_linrec_fwd(f, x, checkpoints=kept)
    g = binding.ssm_linrec_bwd(f, x, dy, checkpoints=kept)
    edge = 2 ** 31 // dim
    for a in (0, edge - 300, n - m):
        # 200 steps away from either cut
        lo, hi = 0 if a == 0 else 200, m if a == n - m else 400
        c = [to64(t[:, a:a + m]) for t in (f, x, dy)]
        y_ref, fin_ref, _ = P.linrec_fwd(c[0], c[1])
        near_linrec(y[:, a + lo:a + hi], y_ref[:, lo:hi], "y", 1e-5)
        df, dx, _, dh0 = P.linrec_bwd(*c)
        near_linrec(g["df"][:, a + lo:a + hi], df[:, lo:hi], "df", 2e-5)
        near_linrec(g["dx"][:, a + lo:a + hi], dx[:, lo:hi], "dx", 2e-5)
        if a == 0:
            near_linrec(g["dinitial_state"], dh0, "dinitial_state", 2e-5)
    near_linrec(fin, fin_ref, "final", 1e-5)


@pytest.mark.parametrize("tokens", [8, 130])
def test_vocab_ce(tokens):
    dim = 2048
    vocab = (2 ** 31 + 2 ** 25) // dim + 3
    randn = _randn(3)
    h, W = randn(tokens, dim), randn(vocab, dim).mul_(3 / dim ** 0.5)
    t = torch.randint(0, vocab, (tokens,), device="cuda")
    t[0], t[1], t[2] = vocab - 1, 0, 2 ** 31 // dim
    loss, lse = binding.ssm_vocab_ce_fwd(h, W, t)
    d = torch.rand(tokens, device="cuda") + 0.1
    g = binding.ssm_vocab_ce_bwd(h, W, t, lse, d, grad_dtype=F32)
    pieces = [slice(v, min(v + 65536, vocab)) for v in range(0, vocab, 65536)]
    ref = torch.logsumexp(torch.stack([torch.logsumexp(h.double() @ W[p].double().t(), -1)
                                       for p in pieces]), 0)
    assert (lse.double() - ref).abs().max() <= 1e-5 * ref.max()
    at = (h.double() * W[t].double()).sum(-1)
    assert (loss.double() - (ref - at)).abs().max() <= 1e-5 * ref.max()
    dh, spread = (torch.zeros(tokens, dim, dtype=torch.float64, device="cuda") for _ in range(2))
    largest = 0.0  # of dW so far
    for p in pieces:
        w64 = W[p].double()
        prob = torch.exp(h.double() @ w64.t() - ref[:, None])
        rows = ((t >= p.start) & (t < p.stop)).nonzero().squeeze(-1)
        prob[rows, t[rows] - p.start] -= 1
        prob *= d.double()[:, None]
        dh += prob @ w64
        spread += prob.square() @ w64.square()
        dw = prob.t() @ h.double()
        largest = max(largest, float(dw.abs().max()))
        if p is pieces[0] or p is pieces[-1] or p.start <= 2 ** 31 // dim < p.stop:
            lim = 6 * 2.0 ** -9 * (prob.square().t() @ h.double().square()).sqrt()
            over = (g["dW"][p].double() - dw).abs() - lim - 1e-5 * largest
            assert float(over.max()) <= 0, p
    lim = 6 * 2.0 ** -9 * spread.sqrt() + 1e-5 * dh.abs().max()
    assert float(((g["dh"].double() - dh).abs() - lim).max()) <= 0
