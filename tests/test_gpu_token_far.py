"""Tensors of more than 2^31 elements: what lies past there is found."""
import pytest

import tok_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spectral_optimizer_ssm_amd as mu
    mu.lib()
    return mu


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\n[case] {request.node.nodeid}", flush=True)
    yield
    torch.cuda.empty_cache()


def close(got, want):
    """bfloat16: half a step, and what float32 leaves."""
    err = (got.double().cpu() - want).abs()
    assert (err <= 2.0**-8 * want.abs() + 1e-5 * want.abs().max()).all(), float(err.max())


@pytest.mark.parametrize("tokens", [100, 3000])
def test_embedding(mu, tokens):
    vocab, n = 2_900_000, 768
    gen = torch.Generator().manual_seed(1)
    table = torch.empty(vocab, n, dtype=BF16, device="cuda").normal_()
    ids = torch.cat([torch.randint(vocab - 50, vocab, (tokens - 50,), generator=gen), torch.randint(0, 50, (50,), generator=gen)])
    y = mu.muon_embedding(table, ids.cuda())
    assert torch.equal(y, table[ids.cuda()])
    dy = torch.randn(tokens, n, generator=gen).to(BF16)
    del table
    d = mu.muon_embedding_backward(dy.cuda(), ids.cuda(), vocab, dtype=BF16)
    near, _ = ref.embedding_grad(dy, ids, 50)
    far, _ = ref.embedding_grad(dy, ids - (vocab - 50), 50)
    close(d[:50], near)
    close(d[-50:], far)
    assert not any(bool(part.any()) for part in d[50:-50].split(300_000))


def test_logprobs(mu):
    rows, vocab = 43_000, 50_280
    x = torch.empty(rows, vocab, dtype=BF16, device="cuda").normal_(std=3.0)
    ids = torch.arange(rows, device="cuda") % vocab
    logp, H, stats, top_ids, top_logp = mu.muon_token_logprobs(x, ids, top=3)
    some = torch.tensor([0, 1, 42_710, 42_711, 42_998, 42_999])
    xs = x[some.cuda()].cpu()
    want = ref.logprobs(xs, ids.cpu()[some], top=3)
    at = some.cuda()
    # a few hundred roundings of 2^-24 of numbers below 30
    assert float((logp[at].cpu().double() - want["logp"]).abs().max()) < 1e-4
    assert float((H[at].cpu().double() - want["entropy"]).abs().max()) < 1e-4
    assert torch.equal(top_ids[at].cpu(), want["top_ids"])
    dl = torch.linspace(-1.0, 1.0, rows, device="cuda")
    grad, _ = ref.logprobs_grad(xs, ids.cpu()[some], stats[at].cpu(), dl[at].cpu())
    mu.muon_token_logprobs_backward(x, ids, stats, dl, dlogits=x)
    close(x[at], grad)


def test_group_norm(mu):
    rows, n = 1_450_000, 1536
    x, z = (torch.empty(rows, n, dtype=BF16, device="cuda").normal_() for _ in range(2))
    w = torch.rand(n, device="cuda")
    y, _, rstd = mu.muon_group_norm(x, 8, w, gate=z)
    at = torch.tensor([0, 1, rows - 2, rows - 1], device="cuda")
    xs, zs = x[at].cpu(), z[at].cpu()
    close(y[at], ref.group_norm(xs, 8, w.cpu(), z=zs)[0])
    dx, dz, _, _ = mu.muon_group_norm_backward(y, x, 8, w, None, None, rstd, gate=z)
    want = ref.group_norm_grads(y[at].cpu(), xs, 8, w.cpu(), None, None, rstd[at].cpu(), zs)
    close(dx[at], want[0])
    close(dz[at], want[1])
