"""The operators together, as the example's language model runs them: its loss and
every gradient against the same model in plain fp64 autograd, its single-token
steps against the whole sequence, and a falling loss.

Tolerances: activations are bf16 (2^-9 relative each) through two layers of four
rounded tensors and back again, independent roundings: the gradients' relative
2-norm error is a few times 2^-8, taken as 5e-2; the loss, a mean over tokens, 1e-2."""
import pytest
import torch

from examples import recurrent_lm as ex

pytestmark = pytest.mark.gpu


def _plain_loss(model, params, tokens, targets):
    """The model in fp64 on the same parameter values."""
    emb, norm, layers = params
    x = emb[tokens]
    stream = torch.zeros_like(x)

    def rms(s, w):
        return s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-5) * w

    for nw, into, back in layers:
        stream = stream + x
        f, v, z = (rms(stream, nw) @ into).chunk(3, -1)
        a, h, hs = torch.sigmoid(f), torch.zeros_like(v[:, 0]), []
        for t in range(v.shape[1]):
            h = a[:, t] * h + (1 - a[:, t]) * v[:, t]
            hs.append(h)
        x = (torch.stack(hs, 1) * z * torch.sigmoid(z)) @ back
    logits = rms(stream + x, norm) @ emb.t()
    return torch.nn.functional.cross_entropy(logits.reshape(-1, logits.shape[-1]),
                                             targets.reshape(-1), ignore_index=-100)


def test_loss_and_gradients_match_the_plain_model():
    model = ex.RecurrentLM(vocab=97, dim=64, layers=2, seed=3)
    rng = torch.Generator().manual_seed(4)
    tokens, targets = ex.batch_of(rng, 3, 83, 97, "cuda")
    loss = model.loss(tokens, targets)
    loss.backward()
    # the example rounds its matrices to bf16 where it uses them
    leaf = [p.detach().to(torch.bfloat16).double().requires_grad_() if p.dim() == 2 else
            p.detach().double().requires_grad_() for p in model.parameters()]
    layers = [tuple(leaf[2 + 3 * i:5 + 3 * i]) for i in range(2)]
    ref = _plain_loss(model, (leaf[0], leaf[1], layers), tokens, targets)
    ref.backward()
    assert abs(loss.item() - ref.item()) < 1e-2 * ref.item()
    for p, r in zip(model.parameters(), leaf):
        err = ((p.grad.double() - r.grad).norm() / r.grad.norm()).item()
        assert err < 5e-2, (tuple(p.shape), err)


@pytest.mark.parametrize("eight_bit", [False, True])
def test_single_tokens_match_the_whole_sequence(eight_bit):
    """The loss of the tokens' logits, one token at a time with the states carried,
    against the training forward (1e-2; with 8-bit norms, 3 mantissa bits, 5e-2)."""
    model = ex.RecurrentLM(vocab=97, dim=64, layers=2, seed=5)
    rng = torch.Generator().manual_seed(6)
    tokens, targets = ex.batch_of(rng, 3, 40, 97, "cuda")
    whole = float(model.loss(tokens, targets).detach())
    states = model.states(3)
    logits = torch.stack([model.step(tokens[:, t], states, eight_bit) for t in range(40)], 1)
    steps = float(torch.nn.functional.cross_entropy(logits.double().reshape(-1, 97),
                                                    targets.reshape(-1), ignore_index=-100))
    assert abs(steps - whole) < (5e-2 if eight_bit else 1e-2) * whole


def test_training_learns():
    first, last = ex.main(steps=60)
    assert last < 0.5 * first, (first, last)
