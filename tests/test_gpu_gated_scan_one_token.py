"""Rows of a single token through the forward and backward calls, whose token
stride says nothing: as rows of their own, as a token of longer tensors, and at
any element."""
import pytest

from test_gpu_gated_scan import BF16, F32, _announce, check_backward, check_forward, inputs, mu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 2, 1, 64, 128), (5, 1, 4, 2, 80, 64), (3, 1, 2, 2, 17, 9)], ids=str)
def test_one_token(mu, shape, dtype):
    x = inputs(*shape, dtype, seed=81)
    check_forward(mu, x)
    check_backward(mu, x)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off", [0, 1, 3])
@pytest.mark.parametrize("shape", [(4, 1, 4, 2, 64, 128), (2, 1, 3, 1, 40, 72)], ids=str)
def test_one_token_of_longer_tensors(mu, shape, off, dtype):
    """The last token of a longer tensor, up to the end of its memory."""
    B, _, H, G, P, N = shape
    x = {n: t.cuda() for n, t in inputs(*shape, dtype, seed=82).items()}

    def last(t):
        long = torch.full((B, 3, off + t[0, 0].numel()), float("nan"), dtype=t.dtype, device="cuda")
        long[:, 2, off:] = t.flatten(1)
        return long[:, 2:, off:].unflatten(2, t.shape[2:])

    rest = dict(gate=x["b"], S0=x["S0"])
    want = mu.muon_gated_scan(x["v"], x["k"], x["q"], x["g"], **rest)
    grads = mu.muon_gated_scan_backward(x["v"], x["k"], x["q"], x["g"], x["dy"], dS=x["dS"], **rest)
    z = {n: last(x[n]) for n in ("v", "k", "q", "g", "b", "dy")}
    rest["gate"] = z["b"]
    got = mu.muon_gated_scan(z["v"], z["k"], z["q"], z["g"], **rest)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = mu.muon_gated_scan_backward(z["v"], z["k"], z["q"], z["g"], z["dy"], dS=x["dS"], **rest)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
