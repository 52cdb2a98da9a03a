"""A Mamba-2 style block trained with this library: root-mean-square norm, input
projection, gated scan, output projection; Muon on the two projections, AdamW on
the rest, then the trained block run token by token as a decoder would.

    python examples/mamba_block.py [--steps 60]

The block learns to reproduce a fixed random block of the same shape (a
teacher) on random sequences; the loss is printed as it falls, and at the end
the largest difference between decoding and the scan over the whole sequence.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spectral_optimizer_ssm_amd as mu  # noqa: E402

D, HEADS, P, N = 256, 8, 64, 128
INNER = HEADS * P


class RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        y, _, rstd = mu.muon_layer_norm(x, w, center=False)
        ctx.save_for_backward(x, w, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, rstd = ctx.saved_tensors
        dx, dw, _ = mu.muon_layer_norm_backward(dy.contiguous(), x, w, None, rstd, center=False, bias_grad=False)
        return dx, dw


class GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, v, k, q, log_decay, gate):
        ctx.save_for_backward(v, k, q, log_decay, gate)
        return mu.muon_gated_scan(v, k, q, log_decay, gate=gate)[0]

    @staticmethod
    def backward(ctx, dy):
        v, k, q, log_decay, gate = ctx.saved_tensors
        return mu.muon_gated_scan_backward(v, k, q, log_decay, dy.contiguous(), gate=gate)[:5]


class Block:
    """Parameters are float32; activations and products bfloat16."""

    def __init__(self, gen):
        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen) * scale).cuda().requires_grad_()

        self.w_in = normal(INNER + 2 * N + HEADS, D, scale=D ** -0.5)
        self.w_out = normal(D, INNER, scale=INNER ** -0.5)
        self.norm = torch.ones(D, device="cuda", requires_grad=True)
        self.dt_bias = torch.full((HEADS,), -3.0, device="cuda", requires_grad=True)
        self.a_log = torch.log(torch.arange(1.0, HEADS + 1)).cuda().requires_grad_()

    def project(self, h):
        """v, k, q (column ranges of one tensor), log decays and input gates."""
        z = h @ self.w_in.to(h.dtype).T
        v, k, q, dt = z.split([INNER, N, N, HEADS], dim=-1)
        dt = torch.nn.functional.softplus(dt.float() + self.dt_bias)
        return v.unflatten(-1, (HEADS, P)), k.unsqueeze(-2), q.unsqueeze(-2), -dt * torch.exp(self.a_log), dt

    def out(self, x, y):
        return x + y.flatten(-2) @ self.w_out.to(y.dtype).T

    def __call__(self, x):
        return self.out(x, GatedScan.apply(*self.project(RmsNorm.apply(x, self.norm))))

    @torch.no_grad()
    def decode(self, x, state):
        """One token a sequence: x [batch, D]; the state is moved on in place."""
        v, k, q, log_decay, dt = self.project(mu.muon_layer_norm(x, self.norm, center=False)[0])
        y, _ = mu.muon_gated_scan_step(v, k, q, log_decay, state, gate=dt)
        return self.out(x, y)


def train(steps=60, batch=4, tokens=300, seed=0, log=print):
    """Losses of the steps and the block."""
    gen = torch.Generator().manual_seed(seed)
    teacher, block = Block(gen), Block(gen)
    muon, rest = [block.w_in, block.w_out], [block.norm, block.dt_bias, block.a_log]
    momentum = [torch.zeros_like(w) for w in muon]
    moments = [[torch.zeros_like(w) for w in rest] for _ in range(2)]
    ws, losses = None, []
    for step in range(1, steps + 1):
        x = torch.randn(batch, tokens, D, generator=gen).cuda().bfloat16()
        with torch.no_grad():
            target = teacher(x).float()
        loss = (block(x).float() - target).square().mean()
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
    return losses, block


@torch.no_grad()
def decode_difference(block, batch=3, tokens=40, seed=1):
    """Largest difference between decoding and the scan, relative to the outputs' size."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(batch, tokens, D, generator=gen).cuda().bfloat16()
    want = block(x)
    state = torch.zeros(batch, HEADS, P, N, device="cuda")
    got = torch.stack([block.decode(x[:, t], state) for t in range(tokens)], 1)
    return float((got.float() - want.float()).abs().max() / want.float().square().mean().sqrt())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    losses, block = train(ap.parse_args().steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    print(f"decoding against the scan: {decode_difference(block):.4f} of the outputs' size")
