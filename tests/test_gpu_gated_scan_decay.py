"""The gradient of the log decays under strong decay, where the pairs of tokens
that cross a token weigh far less than those that do not.

dg_t = e^{g_t} <D_t, S_{t-1}> with D_t the gradient of the state after t.  What a
float32 computation of it can lose is relative to e^{g_t} sum |D_t| |S_{t-1}|:
tokens are compared one by one within F32_TOL of that, and the whole tensor
within F32_TOL of its own norm (decays that are all equal leave the nearest pair
alone, so nothing cancels in it but its two dot products)."""
import pytest

import seq_reference as ref
from test_gpu_gated_scan import BF16, F32, F32_TOL, _announce, backward, inputs, mu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def sizes(x):
    """e^{g_t} sum |D_t| |S_{t-1}| of every token and head, in float64."""
    _, _, states = ref.scan(x["v"], x["k"], x["q"], x["g"], x["b"], x["S0"], keep=True)
    H, G = x["v"].shape[2], x["k"].shape[2]
    k, q = (x[n].double().repeat_interleave(H // G, 2) for n in ("k", "q"))
    a, dy = torch.exp(x["g"].double()), x["dy"].double()
    D = torch.zeros_like(states[0]) if x["dS"] is None else x["dS"].double()
    out = torch.zeros_like(a)
    for t in reversed(range(a.shape[1])):
        D = D + dy[:, t, :, :, None] * q[:, t, :, None, :]
        out[:, t] = a[:, t] * (D.abs() * states[t].abs()).sum((2, 3))
        D = a[:, t, :, None, None] * D
    return out


def check(mu, x, whole):
    got = backward(mu, x)[3].cpu().double()
    want = ref.scan_grads(x["v"], x["k"], x["q"], x["g"], x["dy"], x["b"], x["S0"], x["dS"])[3]
    worst = float(((got - want).abs() / sizes(x).clamp_min(1e-300)).max())
    print(f"[parity] dg {ref.rel(got, want):.2e}, worst token {worst:.2e} of its terms", flush=True)
    assert worst <= F32_TOL
    if whole:
        assert ref.rel(got, want) <= F32_TOL


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 300, 2, 1, 64, 128), (2, 50, 4, 2, 40, 72), (1, 130, 2, 1, 130, 64)], ids=str)
@pytest.mark.parametrize("log_decay", [-1.0, -8.0, -20.0])
def test_every_token_decays_strongly(mu, log_decay, shape, dtype):
    x = inputs(*shape, dtype, seed=31)
    x["g"] = torch.full_like(x["g"], log_decay)
    check(mu, x, True)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("token", [0, 1, 15, 16, 37, 63, 64, 127, 128, 200])
def test_one_strong_decay_among_weak_ones(mu, token, dtype):
    x = inputs(1, 260, 2, 1, 64, 128, dtype, seed=32)
    x["g"][:, token] = -25.0
    check(mu, x, False)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_growth_after_a_decay_that_leaves_nothing(mu, dtype):
    """e^-88.5 is 0 in float32, but what follows makes up for it (token 40 brings
    nothing of its own, which that growth would take past float32)."""
    x = inputs(1, 90, 2, 1, 64, 128, dtype, seed=33)
    x["g"][:, 40], x["g"][:, 41] = -88.5, 70.0
    x["b"][:, 40] = 0.0
    check(mu, x, False)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_mixed_decays(mu, dtype):
    """Log decays over four orders of magnitude, next to each other."""
    x = inputs(2, 280, 4, 2, 64, 128, dtype, seed=34)
    gen = torch.Generator().manual_seed(35)
    x["g"] = -torch.exp(torch.rand(x["g"].shape, generator=gen) * 9.2 - 6.0)
    check(mu, x, False)
