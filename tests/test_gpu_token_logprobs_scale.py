"""Token log probabilities at the ends of the temperatures: next to none of it, where the
largest logits share all, and next to nothing but it, where all tokens are alike."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(3, 300), (2, 50_280)])
def test_ends(rows, vocab, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spectral_optimizer_ssm_amd as mu
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=gen, device="cuda").clamp_(max=2.0).to(dtype)
    x[0, 7] = 9.0
    x[1, 5] = x[1, 250] = 9.0
    ids = torch.tensor([7, 250, 1][:rows], device="cuda")
    dl, dh = torch.full((rows,), -1e-3, device="cuda"), torch.zeros(rows, device="cuda")
    logp, H, stats, top, top_logp = mu.muon_token_logprobs(x, ids, scale=2.35e38, top=2)
    half = math.log(0.5)
    assert logp[0] == 0 and H[0] == 0 and top[0, 0] == 7 and top_logp[0, 0] == 0
    assert abs(float(logp[1]) - half) < 1e-6 and abs(float(H[1]) + half) < 1e-6 and top[1].tolist() == [5, 250]
    dx = mu.muon_token_logprobs_backward(x, ids, stats, dl, scale=2.35e38, entropy=H, dentropy=dh)
    assert (dx[0] == 0).all()      # p is 1 at the token and 0 elsewhere
    want = 2.35e35 * 0.5
    assert abs(float(dx[1, 5]) / want - 1) < 2.0**-7 and abs(float(dx[1, 250]) / -want - 1) < 2.0**-7
    assert int((dx[1] != 0).sum()) == 2
    logp, H, stats, _, _ = mu.muon_token_logprobs(x, ids, scale=1e-30)
    # log vocab, from a sum of ones that is exact
    assert torch.allclose(logp, torch.full_like(logp, -math.log(vocab)), rtol=4 * 2.0**-24, atol=0)
    assert torch.allclose(H, torch.full_like(H, math.log(vocab)), rtol=4 * 2.0**-24, atol=0)
