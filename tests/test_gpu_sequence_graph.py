"""Decoding and training steps of the sequence operators in a HIP graph: captured
once, replayed on new inputs with eager work between, every replay against the
eager call."""
import pytest

from test_gpu_gated_scan import BF16, F32, _announce, inputs, mu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch", [1, 300])
def test_single_tokens(mu, batch, dtype):
    """The state moves on in place from replay to replay."""
    def token(seed):
        x = inputs(batch, 1, 4, 2, 64, 128, dtype, seed=seed)
        return {n: x[n][:, 0].cuda() for n in ("v", "k", "q", "g", "b")}, x["S0"].cuda()

    c, S = token(91)
    Y = torch.empty_like(c["v"])
    step = lambda c, S, **kw: mu.muon_gated_scan_step(c["v"], c["k"], c["q"], c["g"], S, gate=c["b"], **kw)  # noqa: E731
    step(c, S, Y=Y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, S, Y=Y)
    eager = S.clone()
    for seed in range(92, 97):
        z, _ = token(seed)
        for n in c:
            c[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        want, _ = step(z, eager)
        torch.cuda.synchronize()
        assert torch.equal(Y, want) and torch.equal(S, eager), seed


def test_norm_forward_and_backward(mu):
    gen = torch.Generator().manual_seed(98)
    draw = lambda: [torch.randn(2000, 768, generator=gen).to(BF16).cuda() for _ in range(2)]  # noqa: E731
    (X, dY), w = draw(), torch.randn(768, generator=gen).cuda()
    ws = torch.empty(mu.lib().muon_layer_norm_backward_workspace_size(2000, 768, mu.MUON_BF16), dtype=torch.uint8, device="cuda")

    def call():
        Y, mean, rstd = mu.muon_layer_norm(X, w)
        return (Y, mean, rstd) + mu.muon_layer_norm_backward(dY, X, w, mean, rstd, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(4):
        a, b = draw()
        X.copy_(a)
        dY.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(got, want))
