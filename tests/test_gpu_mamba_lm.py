"""The operators of a language model together: the example model runs, its gradients
are those of its loss, and a chain of them agrees with float64 autograd of the plain
forms."""
import importlib.util
import os

import pytest

import tok_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F64 = torch.float64


@pytest.fixture(scope="module")
def mu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spectral_optimizer_ssm_amd as mu
    mu.lib()
    return mu


@pytest.fixture(scope="module")
def example(mu):
    spec = importlib.util.spec_from_file_location("mamba_lm", os.path.join(ROOT, "examples", "mamba_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs(example):
    losses, model = example.train(steps=3, batch=4, tokens=65, log=lambda s: None)
    assert len(losses) == 3 and all(torch.isfinite(torch.tensor(losses)))
    text = example.texts(torch.Generator().manual_seed(2), 3, 40)[:, :30]
    ids, logp, entropy = model.next_tokens(text, top=7)
    assert ids.shape == logp.shape == (3, 7) and entropy.shape == (3,)
    assert (ids >= 0).all() and (ids < example.VOCAB).all()
    assert (logp[:, 1:] <= logp[:, :-1]).all() and (logp <= 0).all() and (entropy > 0).all()


@pytest.mark.parametrize("name", ["table", "w_in", "w_out", "mixer_norm", "norm_f"])
def test_example_gradients_against_differences(example, name):
    """Along the gradient itself, so that the difference is as large as can be.  With
    float32 activations the loss (about 5) is off by about 2^-24 x 5 x 10; a step of h
    along the gradient's direction changes it by 2 h |g|, chosen to be 1e-2, and the third
    derivative's part is of the order of (h / |w|)^2 of it."""
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(7)
    model = example.Model(gen, torch.float32)
    text = example.texts(gen, 4, 70)
    p = getattr(model, name)
    p = p[0] if isinstance(p, list) else p
    g, = torch.autograd.grad(model.loss(text), [p])
    size = float(g.double().norm())
    assert size > 0
    h = min(0.5e-2 / size, 0.02 * float(p.detach().norm()))
    with torch.no_grad():
        d = g / size
        p += h * d
        up = float(model.loss(text))
        p -= 2 * h * d
        down = float(model.loss(text))
    got = (up - down) / (2 * h)
    print(f"[case] {name}: |g| {size:.4e}, difference {got:.4e}, step {h:.2e}", flush=True)
    assert abs(got - size) <= 0.02 * size + 1e-5 / h


def test_chain_against_float64(mu):
    """Embedding, gated group norm, a tied output product (torch's) and the loss with an
    entropy bonus, in float32: the gradients of the table (both uses, the second
    accumulated) and of the norm's operands.  Each step is off by what its own test allows;
    together a few times 1e-5 of the largest entry."""
    gen = torch.Generator().manual_seed(12)
    V, n, groups, scale = 500, 96, 4, 1.7
    text = torch.randint(-1, V, (5, 41), generator=gen)
    table, w = 0.3 * torch.randn(V, n, generator=gen), 1.0 + 0.2 * torch.randn(n, generator=gen)
    z = torch.randn(5, 40, n, generator=gen)
    ids, targets = text[:, :-1], text[:, 1:]
    # float64, by autograd
    t64, w64, z64 = (a.to(F64).requires_grad_() for a in (table, w, z))
    x = ref.embedding(t64, ids, scale)
    y = ref.group_norm(x, groups, w64, z=z64)[0]
    lp = torch.log_softmax((y @ t64.T).reshape(-1, V), 1)
    flat = targets.reshape(-1)
    chosen = torch.where(flat >= 0, lp.gather(1, flat.clamp(min=0)[:, None])[:, 0], 0.0)
    H = -(lp.exp() * lp).sum(1)
    loss = -chosen.sum() / 100 - 0.05 * H.sum() / 100
    want = torch.autograd.grad(loss, (t64, w64, z64))
    # the operators
    tg, wg, zg, dev = table.cuda(), w.cuda(), z.cuda(), text.cuda()
    ids, targets = dev[:, :-1], dev[:, 1:]
    x = mu.muon_embedding(tg, ids, scale=scale)
    y, _, rstd = mu.muon_group_norm(x, groups, wg, gate=zg)
    logits = (y.reshape(-1, n) @ tg.T).reshape(5, 40, V)
    logp, entropy, stats, _, _ = mu.muon_token_logprobs(logits, targets)
    got_loss = float(-logp.double().sum() / 100 - 0.05 * entropy.double().sum() / 100)
    loss = float(loss.detach())
    assert abs(got_loss - loss) < 1e-4 * abs(loss)
    one = lambda v: torch.full((1, 1), v, device="cuda").expand(5, 40)  # noqa: E731
    dl = mu.muon_token_logprobs_backward(logits, targets, stats, one(-0.01), entropy=entropy, dentropy=one(-0.0005), dlogits=logits)
    dtable = dl.reshape(-1, V).T @ y.reshape(-1, n)
    dx, dz, dw, _ = mu.muon_group_norm_backward((dl.reshape(-1, V) @ tg).reshape(5, 40, n), x, groups, wg, None, None, rstd, gate=zg)
    mu.muon_embedding_backward(dx, ids, V, scale=scale, dtable=dtable, accumulate=True)
    for name, a, b in (("table", dtable, want[0]), ("w", dw, want[1]), ("z", dz, want[2])):
        err = float((a.double().cpu() - b).abs().max() / b.abs().max())
        print(f"[case] {name}: {err:.2e}", flush=True)
        assert err < 1e-4, name
