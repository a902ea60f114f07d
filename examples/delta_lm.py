"""A small language model whose layers keep a matrix of associations a head: training steps,
then one token at a time.

    python examples/delta_lm.py

Each layer is pre-norm: the residual's addition and RMS norm, one projection to queries, keys
and values, the norm of their heads with the rotation by position, the gated delta rule, and
a projection back; a second, narrow projection gives each head its gate and its step.  The
head is the norm and the cross entropy against the (tied) embedding.  Sequences of a batch
may be shorter than it: a negative token is padding, which no state learns from (its step is
0) or forgets at (its gate is 0).
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import state_space_model_selective_gb300 as ssm  # noqa: E402
from examples.recurrent_lm import AddNorm, VocabLoss, batch_of  # noqa: E402


class QkNorm(torch.autograd.Function):
    """The heads of q and k normed and turned; ``fixed`` is what takes no gradient."""

    @staticmethod
    def forward(ctx, q, k, q_weight, fixed):
        ctx.save_for_backward(q, k, q_weight)
        ctx.fixed = fixed
        return ssm.ssm_qk_norm_rope_fwd(q, k, q_weight=q_weight, **fixed)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, q_weight = ctx.saved_tensors
        g = ssm.ssm_qk_norm_rope_bwd(dq.contiguous(), dk.contiguous(), q, k, q_weight=q_weight,
                                     **ctx.fixed)
        return g["dq"], g["dk"], g["dq_weight"], None


class GatedDelta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        b, n, h, dv = v.shape
        size = ssm.ssm_gated_delta_checkpoint_bytes(b, n, h, q.shape[-1], dv)
        kept = torch.empty(size, dtype=torch.uint8, device=q.device)
        y, _ = ssm.ssm_gated_delta_fwd(q, k, v, g, beta, checkpoints=kept,
                                       return_final_state=False)
        ctx.save_for_backward(q, k, v, g, beta, kept)
        return y

    @staticmethod
    def backward(ctx, dy):
        *five, kept = ctx.saved_tensors
        g = ssm.ssm_gated_delta_bwd(*five, dy.contiguous(), checkpoints=kept,
                                    want_dinitial_state=False)
        return tuple(g[name] for name in ("dq", "dk", "dv", "dg", "dbeta"))


class DeltaLM:
    def __init__(self, vocab=1000, dim=256, layers=2, heads=4, groups=2, dstate=64, headdim=64,
                 seed=0, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def randn(*shape, std):
            return (std * torch.randn(*shape, generator=gen, device=device)).requires_grad_()

        def ones(n, value=1.0):
            return torch.full((n,), value, device=device)

        self.dim, self.device = dim, device
        self.heads, self.groups, self.dstate, self.headdim = heads, groups, dstate, headdim
        self.embedding = randn(vocab, dim, std=dim ** -0.5)
        wide = 2 * groups * dstate + heads * headdim
        self.layers = [{"norm": ones(dim).requires_grad_(),
                        "q_norm": ones(dstate, dstate ** -0.5).requires_grad_(),
                        "into": randn(dim, wide, std=dim ** -0.5),
                        "gates": randn(dim, 2 * heads, std=dim ** -0.5),
                        "back": randn(heads * headdim, dim, std=(heads * headdim) ** -0.5)}
                       for _ in range(layers)]
        self.norm = ones(dim).requires_grad_()
        # keys have length one, so that what a step learns is never too much
        self.k_norm = ones(dstate, dstate ** -0.5)
        self.inv_freq = 1e4 ** -(torch.arange(dstate // 4, device=device, dtype=torch.float64) /
                                 (dstate // 4))

    def parameters(self):
        return [self.embedding, self.norm] + [p for layer in self.layers for p in layer.values()]

    def _inputs(self, n, layer, positions, padding):
        """q, k, v (ranges of one projection), gates and steps, and the norm's arguments."""
        at = self.groups * self.dstate
        wide = n @ layer["into"].to(n.dtype)
        q, k = (wide[..., i * at:(i + 1) * at].unflatten(-1, (self.groups, self.dstate))
                for i in range(2))
        v = wide[..., 2 * at:].unflatten(-1, (self.heads, self.headdim))
        f, b = (n.float() @ layer["gates"]).chunk(2, -1)
        g = -torch.nn.functional.softplus(f - 2).masked_fill(padding, 0)
        beta = torch.sigmoid(b).masked_fill(padding, 0)
        fixed = {"k_weight": self.k_norm, "positions": positions, "inv_freq": self.inv_freq}
        return q, k, v, g, beta, fixed

    def loss(self, tokens, targets):
        """Mean loss over the targets that are not negative.  tokens, targets:
        (batch, seqlen)."""
        W = self.embedding.to(torch.bfloat16)
        padding = (tokens < 0)[..., None]
        x = W[tokens.clamp(min=0)]
        stream = torch.zeros(x.shape, device=x.device)
        positions = torch.arange(tokens.shape[1], device=x.device).expand(tokens.shape).contiguous()
        for layer in self.layers:
            n, stream = AddNorm.apply(x, stream, layer["norm"])
            q, k, v, g, beta, fixed = self._inputs(n, layer, positions, padding)
            q, k = QkNorm.apply(q, k, layer["q_norm"], fixed)
            y = GatedDelta.apply(q, k, v, g, beta)
            x = y.flatten(2) @ layer["back"].to(y.dtype)
        n, _ = AddNorm.apply(x, stream, self.norm)
        flat = targets.reshape(-1)
        per_token = VocabLoss.apply(n.reshape(-1, self.dim), W, flat)
        return per_token.sum() / (flat >= 0).sum().clamp(min=1)

    @torch.no_grad()
    def step(self, tokens, position, states):
        """The next tokens (batch, n; one, or a few drafted ones) from ``position`` (batch,) on:
        logits (batch, n, vocab).  ``states`` (a list of (batch, heads, headdim, dstate) fp32
        tensors) are updated in place."""
        W = self.embedding.to(torch.bfloat16)
        padding = (tokens < 0)[..., None]
        x = W[tokens.clamp(min=0)]
        stream = torch.zeros(x.shape, device=x.device)
        positions = position[:, None] + torch.arange(tokens.shape[1], device=x.device)
        for layer, state in zip(self.layers, states):
            n, _ = ssm.ssm_add_rmsnorm_fwd(x, layer["norm"], stream, sum_out=stream)
            q, k, v, g, beta, fixed = self._inputs(n, layer, positions, padding)
            q, k = ssm.ssm_qk_norm_rope_fwd(q, k, q_weight=layer["q_norm"], **fixed)
            y, _ = ssm.ssm_gated_delta_fwd(q, k, v, g, beta, initial_state=state,
                                           final_state=state)
            x = y.flatten(2) @ layer["back"].to(y.dtype)
        return ssm.ssm_add_rmsnorm_fwd(x, self.norm, stream, sum_out=stream)[0] @ W.t()

    def states(self, batch):
        return [torch.zeros(batch, self.heads, self.headdim, self.dstate, device=self.device)
                for _ in self.layers]


def main(steps=60, batch=16, seqlen=128, vocab=64):
    model = DeltaLM(vocab=vocab)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    rng = torch.Generator().manual_seed(1)
    for i in range(steps):
        loss = model.loss(*batch_of(rng, batch, seqlen, vocab, model.device))
        opt.zero_grad()
        loss.backward()
        opt.step()
        if i % 20 == 0 or i == steps - 1:
            print(f"step {i}: loss {float(loss.detach()):.3f}")
    tokens, targets = batch_of(rng, 4, 64, vocab, model.device)
    states, hits = model.states(4), 0
    for t in range(tokens.shape[1]):
        at = torch.full((4,), t, device=tokens.device)
        best = model.step(tokens[:, t:t + 1], at, states)[:, 0].argmax(-1)
        hits += int(((best == targets[:, t]) & (targets[:, t] >= 0)).sum())
    print(f"one token at a time: {hits} of {int((targets >= 0).sum())} next tokens right")


if __name__ == "__main__":
    main()
