"""A small recurrent language model on the library's operators: training steps,
then one token at a time.

    python examples/recurrent_lm.py

Each layer is pre-norm: the residual's addition and RMS norm, one projection to the
recurrence's gate, input and output gate, the gated linear recurrence, and a
projection back; the head is the norm and the cross entropy against the (tied)
embedding, whose logits never exist.  The residual stream is kept in fp32, the
activations in bf16; the projections are torch matrix products.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import state_space_model_selective_gb300 as ssm  # noqa: E402


class AddNorm(torch.autograd.Function):
    """y, s = rmsnorm(x + residual) * weight, x + residual."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        y, s = ssm.ssm_add_rmsnorm_fwd(x, weight, residual)
        ctx.save_for_backward(s, weight)
        ctx.x_dtype = x.dtype
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, weight = ctx.saved_tensors
        g = ssm.ssm_add_rmsnorm_bwd(dy.contiguous(), s, weight, dsum=ds.contiguous(),
                                    x_dtype=ctx.x_dtype)
        return g["dx"], g["dresidual"], g["dweight"]


class LinRec(torch.autograd.Function):
    """h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(f); returns h * silu(z)."""

    @staticmethod
    def forward(ctx, f, x, z):
        b, n, d = x.shape
        kept = torch.empty(ssm.ssm_linrec_checkpoint_bytes(b, n, d) // 4, device=x.device)
        y, _ = ssm.ssm_linrec_fwd(f, x, z, checkpoints=kept, return_final_state=False)
        ctx.save_for_backward(f, x, z, kept)
        return y

    @staticmethod
    def backward(ctx, dy):
        f, x, z, kept = ctx.saved_tensors
        g = ssm.ssm_linrec_bwd(f, x, dy.contiguous(), z, checkpoints=kept,
                               want_dinitial_state=False)
        return g["df"], g["dx"], g["dz"]


class VocabLoss(torch.autograd.Function):
    """Cross entropy of h W^T per token; a negative target carries none."""

    @staticmethod
    def forward(ctx, h, W, targets):
        loss, lse = ssm.ssm_vocab_ce_fwd(h, W, targets)
        ctx.save_for_backward(h, W, targets, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        h, W, targets, lse = ctx.saved_tensors
        g = ssm.ssm_vocab_ce_bwd(h, W, targets, lse, dloss.contiguous())
        return g["dh"], g["dW"], None


class RecurrentLM:
    def __init__(self, vocab=1000, dim=256, layers=2, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape, std):
            return (std * torch.randn(*shape, generator=g, device=device)).requires_grad_()

        self.dim, self.device = dim, device
        self.embedding = randn(vocab, dim, std=dim ** -0.5)
        self.layers = [{"norm": torch.ones(dim, device=device, requires_grad=True),
                        "into": randn(dim, 3 * dim, std=dim ** -0.5),
                        "back": randn(dim, dim, std=dim ** -0.5)} for _ in range(layers)]
        self.norm = torch.ones(dim, device=device, requires_grad=True)

    def parameters(self):
        return [self.embedding, self.norm] + [p for layer in self.layers for p in layer.values()]

    def _gates(self, n, layer):
        f, x, z = (n @ layer["into"].to(n.dtype)).chunk(3, -1)
        return f, x, z  # ranges of one projection: the recurrence reads them where they are

    def loss(self, tokens, targets):
        """Mean loss over the targets that are not negative.  tokens, targets:
        (batch, seqlen)."""
        W = self.embedding.to(torch.bfloat16)
        x = W[tokens]
        stream = torch.zeros(x.shape, device=x.device)
        for layer in self.layers:
            n, stream = AddNorm.apply(x, stream, layer["norm"])
            x = LinRec.apply(*self._gates(n, layer)) @ layer["back"].to(n.dtype)
        n, _ = AddNorm.apply(x, stream, self.norm)
        flat = targets.reshape(-1)
        per_token = VocabLoss.apply(n.reshape(-1, self.dim), W, flat)
        return per_token.sum() / (flat >= 0).sum().clamp(min=1)

    @torch.no_grad()
    def step(self, tokens, states, eight_bit=False):
        """One token for each sequence: logits (batch, vocab); ``states`` (a list of
        (batch, dim) fp32 tensors) are updated in place.  ``eight_bit``: the norms leave
        e4m3 values and one scale a row, as an 8-bit product takes them."""
        W = self.embedding.to(torch.bfloat16)
        x = W[tokens]
        stream = torch.zeros(x.shape, device=x.device)

        def norm(x, stream, weight):
            if not eight_bit:
                return ssm.ssm_add_rmsnorm_fwd(x, weight, stream, sum_out=stream)[0]
            q, scales, _ = ssm.ssm_add_rmsnorm_e4m3_fwd(x, weight, stream, group=0, sum_out=stream)
            return (q.float() * scales).to(x.dtype)

        for layer, state in zip(self.layers, states):
            f, v, z = (t[:, None] for t in self._gates(norm(x, stream, layer["norm"]), layer))
            y, _ = ssm.ssm_linrec_fwd(f, v, z, initial_state=state, final_state=state)
            x = y[:, 0] @ layer["back"].to(x.dtype)
        return norm(x, stream, self.norm) @ W.t()

    def states(self, batch):
        return [torch.zeros(batch, self.dim, device=self.device) for _ in self.layers]


def batch_of(rng, batch, seqlen, vocab, device):
    """Walks over a fixed random permutation of the vocabulary from random starts: the
    next token is known from the present one.  The first two targets carry no loss."""
    after = torch.randperm(vocab, generator=torch.Generator().manual_seed(vocab))
    walk = [torch.randint(0, vocab, (batch,), generator=rng)]
    for _ in range(seqlen):
        walk.append(after[walk[-1]])
    walk = torch.stack(walk, 1).to(device)
    targets = walk[:, 1:].clone()
    targets[:, :2] = -100
    return walk[:, :-1].contiguous(), targets


def main(steps=60, batch=16, seqlen=128, vocab=64):
    model = RecurrentLM(vocab=vocab)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    rng = torch.Generator().manual_seed(1)
    first = last = None
    for i in range(steps):
        loss = model.loss(*batch_of(rng, batch, seqlen, vocab, model.device))
        opt.zero_grad()
        loss.backward()
        opt.step()
        last = float(loss.detach())
        first = last if first is None else first
        if i % 20 == 0 or i == steps - 1:
            print(f"step {i}: loss {last:.3f}")
    tokens, targets = batch_of(rng, 4, 64, vocab, model.device)
    for eight_bit in (False, True):
        states, hits = model.states(4), 0
        for t in range(tokens.shape[1]):
            best = model.step(tokens[:, t], states, eight_bit).argmax(-1)
            hits += int(((best == targets[:, t]) & (targets[:, t] >= 0)).sum())
        print(f"one token at a time{', 8-bit norms' if eight_bit else ''}: {hits} of "
              f"{int((targets >= 0).sum())} next tokens right")
    return first, last


if __name__ == "__main__":
    main()
