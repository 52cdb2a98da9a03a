"""A small Mamba-2 style language model trained with this library and then asked for
its answers: token embedding, blocks of a root-mean-square norm, an input
projection, the gated scan, the gated group norm and an output projection, a tied
output embedding and the log probabilities of the next tokens.  Muon trains the
projections, AdamW the rest.

    python examples/mamba_lm.py [--steps 100]

Each token of the texts has one that mostly follows it; the mean loss is printed, and
at the end what the model takes to be the likeliest next tokens of one text.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import spectral_optimizer_ssm_amd as mu  # noqa: E402
from mamba_block import GatedScan, RmsNorm  # noqa: E402

VOCAB, D, HEADS, P, N, LAYERS = 250, 128, 4, 64, 64, 2
INNER = HEADS * P
PADDING = -1


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, dtype):
        ctx.save_for_backward(ids)
        ctx.vocab = table.shape[0]
        return mu.muon_embedding(table, ids, dtype=dtype)

    @staticmethod
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        return mu.muon_embedding_backward(dy.contiguous(), ids, ctx.vocab), None, None


class GatedNorm(torch.autograd.Function):
    """Root-mean-square norm of x silu(z), each head's channels by themselves."""

    @staticmethod
    def forward(ctx, x, z, w):
        y, _, rstd = mu.muon_group_norm(x, HEADS, w, gate=z)
        ctx.save_for_backward(x, z, w, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, z, w, rstd = ctx.saved_tensors
        return mu.muon_group_norm_backward(dy.contiguous(), x, HEADS, w, None, None, rstd, gate=z)[:3]


class LogProbs(torch.autograd.Function):
    """log p of the tokens, 0 at padding."""

    @staticmethod
    def forward(ctx, logits, tokens):
        logp, _, stats, _, _ = mu.muon_token_logprobs(logits, tokens, entropy=False)
        ctx.save_for_backward(logits, tokens, stats)
        return logp

    @staticmethod
    def backward(ctx, dlogp):
        return mu.muon_token_logprobs_backward(*ctx.saved_tensors, dlogp), None


class Model:
    """Parameters are float32; activations and products `dtype`."""

    def __init__(self, gen, dtype=torch.bfloat16):
        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen) * scale).cuda().requires_grad_()

        self.dtype = dtype
        self.table = normal(VOCAB, D, scale=0.05)
        self.w_in = [normal(2 * INNER + 2 * N + HEADS, D, scale=D ** -0.5) for _ in range(LAYERS)]
        self.w_out = [normal(D, INNER, scale=INNER ** -0.5) for _ in range(LAYERS)]
        ones = lambda n: torch.ones(n, device="cuda", requires_grad=True)  # noqa: E731
        self.norm, self.mixer_norm = [ones(D) for _ in range(LAYERS)], [ones(INNER) for _ in range(LAYERS)]
        self.norm_f = ones(D)
        self.dt_bias = [torch.full((HEADS,), -2.0, device="cuda", requires_grad=True) for _ in range(LAYERS)]
        self.a_log = [torch.log(torch.arange(1.0, HEADS + 1)).cuda().requires_grad_() for _ in range(LAYERS)]

    def muon_parameters(self):
        return self.w_in + self.w_out

    def other_parameters(self):
        return [self.table, self.norm_f, *self.norm, *self.mixer_norm, *self.dt_bias, *self.a_log]

    def logits(self, ids):
        x = Embedding.apply(self.table, ids, self.dtype)
        for i in range(LAYERS):
            h = RmsNorm.apply(x, self.norm[i]) @ self.w_in[i].to(self.dtype).T
            z, v, k, q, dt = h.split([INNER, INNER, N, N, HEADS], dim=-1)
            dt = torch.nn.functional.softplus(dt.float() + self.dt_bias[i])
            y = GatedScan.apply(v.unflatten(-1, (HEADS, P)), k.unsqueeze(-2), q.unsqueeze(-2), -dt * torch.exp(self.a_log[i]), dt)
            x = x + GatedNorm.apply(y.flatten(-2), z, self.mixer_norm[i]) @ self.w_out[i].to(self.dtype).T
        return RmsNorm.apply(x, self.norm_f) @ self.table.to(self.dtype).T

    def loss(self, text):
        """Mean loss of each token after those before it; padding counts for nothing."""
        targets = text[:, 1:]
        logp = LogProbs.apply(self.logits(text[:, :-1]), targets)
        return -logp.sum() / (targets != PADDING).sum()

    @torch.no_grad()
    def next_tokens(self, text, top=5):
        """The likeliest next tokens of each text, their log probabilities, and the entropy."""
        _, entropy, _, ids, logp = mu.muon_token_logprobs(self.logits(text)[:, -1], top=top)
        return ids, logp, entropy


def follower(token):
    return (token * 7 + 3) % VOCAB


def texts(gen, batch, tokens):
    """Nine tokens of ten are the follower of the one before; the last tokens of every other
    text are padding."""
    text = torch.randint(0, VOCAB, (batch, tokens), generator=gen)
    keep = torch.rand(batch, tokens, generator=gen) < 0.9
    for t in range(1, tokens):
        text[:, t] = torch.where(keep[:, t], follower(text[:, t - 1]), text[:, t])
    text[1::2, -(tokens // 8 + 1):] = PADDING
    return text.cuda()


def train(steps=100, batch=8, tokens=129, seed=0, log=print):
    """Losses of the steps and the model."""
    gen = torch.Generator().manual_seed(seed)
    model = Model(gen)
    muon, rest = model.muon_parameters(), model.other_parameters()
    momentum = [torch.zeros_like(w) for w in muon]
    moments = [[torch.zeros_like(w) for w in rest] for _ in range(2)]
    ws, losses = None, []
    for step in range(1, steps + 1):
        loss = model.loss(texts(gen, batch, tokens))
        grads = torch.autograd.grad(loss, muon + rest)
        with torch.no_grad():
            groups = [mu.MuonGroup(W=w.detach()[None], M=m[None], G=g[None].contiguous(), lr=0.02, beta=0.9)
                      for w, m, g in zip(muon, momentum, grads)]
            ws = mu.muon_step(groups, steps=5, workspace=ws)
            mu.muon_adamw([w.detach() for w in rest], [g.contiguous() for g in grads[len(muon):]], *moments, lr=3e-3, step=step,
                          weight_decay=0.0)
        losses.append(float(loss.detach()))
        if step == 1 or step % 10 == 0:
            log(f"step {step:4d}  loss {losses[-1]:.4f}")
    return losses, model


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=100)
    losses, model = train(ap.parse_args().steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    text = texts(torch.Generator().manual_seed(1), 1, 100)
    ids, logp, entropy = model.next_tokens(text)
    print(f"{follower(int(text[0, -1]))} mostly follows; taken to be likeliest, with an entropy of {float(entropy[0]):.2f}:")
    for i, p in zip(ids[0].tolist(), logp[0].tolist()):
        print(f"  {i:4d}  log p {p:.3f}")
