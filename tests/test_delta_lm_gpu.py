"""Norms of heads, the gated delta rule, the residual's norm and the cross entropy together, as
the example's language model runs them: its loss and every gradient against the same model in
plain fp64 autograd, its steps against the whole sequence.

Tolerances: activations are bf16, 2^-9 relative each on average, through two layers of six
rounded tensors and back again: 24 independent roundings, 24^0.5 2^-9 = 1e-2 of a gradient's
2-norm, and up to a few times that where sums of either sign cancel (the gates): 5e-2; the
loss, a mean over tokens, 1e-2."""
import pytest
import torch

from examples import delta_lm as ex

pytestmark = pytest.mark.gpu


def _plain_loss(model, params, tokens, targets):
    """The model in fp64 on the same parameter values."""
    emb, norm, layers = params
    pad = (tokens < 0)[..., None]
    x = emb[tokens.clamp(min=0)]
    stream = torch.zeros_like(x)
    b, n = tokens.shape
    angle = torch.arange(n, device=x.device).double()[:, None] * model.inv_freq
    cos, sin = (t[None, :, None] for t in (torch.cos(angle), torch.sin(angle)))

    def rms(s, w):
        return s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-5) * w

    def turn(t):
        half = cos.shape[-1]
        a, c, rest = t[..., :half], t[..., half:2 * half], t[..., 2 * half:]
        return torch.cat((a * cos - c * sin, a * sin + c * cos, rest), -1)

    ratio, at = model.heads // model.groups, model.groups * model.dstate
    for nw, qw, into, gates, back in layers:
        stream = stream + x
        y = rms(stream, nw)
        wide, (f, s) = y @ into, (y @ gates).chunk(2, -1)
        q, k = (wide[..., i * at:(i + 1) * at].unflatten(-1, (model.groups, -1)) for i in range(2))
        q, k = (turn(rms(t, w)).repeat_interleave(ratio, 2) for t, w in ((q, qw), (k, model.k_norm.double())))
        v = wide[..., 2 * at:].unflatten(-1, (model.heads, -1))
        decay = torch.exp(-torch.nn.functional.softplus(f - 2)).masked_fill(pad, 1)
        beta = torch.sigmoid(s).masked_fill(pad, 0)
        S, ys = torch.zeros(b, model.heads, v.shape[-1], model.dstate, device=x.device).double(), []
        for t in range(n):
            S = S * decay[:, t, :, None, None]
            u = beta[:, t, :, None] * (v[:, t] - (S @ k[:, t, :, :, None])[..., 0])
            S = S + u[..., None] * k[:, t, :, None]
            ys.append((S @ q[:, t, :, :, None])[..., 0])
        x = torch.stack(ys, 1).flatten(2) @ back
    logits = rms(stream + x, norm) @ emb.t()
    return torch.nn.functional.cross_entropy(logits.reshape(-1, logits.shape[-1]),
                                             targets.reshape(-1), ignore_index=-100)


def _leaves(model):
    """The example rounds its matrices to bf16 where it uses them, but for the gates'."""
    fp32 = {id(layer["gates"]) for layer in model.layers}
    leaf = [(p.detach().to(torch.bfloat16) if p.dim() == 2 and id(p) not in fp32 else
             p.detach()).double().requires_grad_() for p in model.parameters()]
    return leaf, [tuple(leaf[2 + 5 * i:7 + 5 * i]) for i in range(len(model.layers))]


def _batch(batch, seqlen, padded):
    rng = torch.Generator().manual_seed(4)
    tokens, targets = ex.batch_of(rng, batch, seqlen, 97, "cuda")
    if padded:  # sequences of other lengths, and one that starts late
        tokens[1, seqlen // 2:], targets[1, seqlen // 2:] = -1, -100
        tokens[2, :7], targets[2, :7] = -1, -100
    return tokens, targets


@pytest.mark.parametrize("padded", [False, True])
def test_loss_and_gradients_match_the_plain_model(padded):
    model = ex.DeltaLM(vocab=97, dim=64, heads=4, groups=2, dstate=32, headdim=24, seed=3)
    tokens, targets = _batch(3, 83, padded)
    loss = model.loss(tokens, targets)
    loss.backward()
    leaf, layers = _leaves(model)
    ref = _plain_loss(model, (leaf[0], leaf[1], layers), tokens, targets)
    ref.backward()
    assert abs(loss.item() - ref.item()) < 1e-2 * ref.item()
    for p, r in zip(model.parameters(), leaf):
        err = ((p.grad.double() - r.grad).norm() / r.grad.norm()).item()
        assert err < 5e-2, (tuple(p.shape), err)


@pytest.mark.parametrize("at_once", [1, 4, 20])
def test_steps_match_the_whole_sequence(at_once):
    """One token at a time, a few, and a run of a prompt (in chunks), the states carried."""
    model = ex.DeltaLM(vocab=97, dim=64, heads=4, groups=2, dstate=32, headdim=24, seed=5)
    tokens, targets = _batch(3, 40, True)
    whole = float(model.loss(tokens, targets).detach())
    states = model.states(3)
    logits = [model.step(tokens[:, t:t + at_once], torch.full((3,), t, device="cuda"), states)
              for t in range(0, 40, at_once)]
    steps = float(torch.nn.functional.cross_entropy(torch.cat(logits, 1).double().reshape(-1, 97),
                                                    targets.reshape(-1), ignore_index=-100))
    assert abs(steps - whole) < 1e-2 * whole


def test_the_example_runs(capsys):
    ex.main(steps=3, batch=2, seqlen=70)
    assert "next tokens right" in capsys.readouterr().out
