"""GPU parity of the token log probabilities, the entropy, the likeliest tokens and
their gradients with the float64 reference (tests/tok_reference.py).

Tolerances, in units of 2^-24.  A row's sum is off by a chain of at most vocab / 256
additions (an element at a time by a thread) and a hundred in the joins, and each of
its exponentials by twice its exponent; so L is off by vocab / 256 + 100 + 4 sum p |t|,
log p by that and 4 |t_id| more, H by the same relative error of sum p |t| and, from
the exponents, 4 sum p t^2.  Gradients: as the size that the reference gives, by 32."""
import math

import pytest

import tok_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0**-8, F32: 0.0}
U = 2.0**-24


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


def same_or_close(got, want, bound):
    """Not finite alike, and otherwise within bound."""
    got = got.double().cpu()
    # past the largest float32 and half a step, a value's rounding is an infinity (1.25 times the lowest one)
    want = torch.where(want.abs() >= float(torch.finfo(F32).max) * (1 + 2.0**-25), torch.sign(want) * math.inf, want)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)])
    over = ((got - want).abs() - bound)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())


def check_forward(mu, x, ids, scale, top, dev=None):
    rows, vocab = x.shape
    sc = float(torch.tensor(scale, dtype=F32))
    want = ref.logprobs(x, ids, sc, top)
    got = mu.muon_token_logprobs(x.cuda() if dev is None else dev, None if ids is None else ids.cuda(), scale=scale, top=top)
    logp, H, stats, top_ids, top_logp = got
    first, second = (torch.nan_to_num(want[k]) for k in ("first", "second"))
    chain = vocab / 256 + 100
    tol_L = U * (chain + 4 * first)
    same_or_close(stats[:, 0], want["stats"][:, 0], torch.zeros(rows, dtype=torch.float64))
    same_or_close(stats[:, 1], want["stats"][:, 1], tol_L)
    same_or_close(H, want["entropy"], tol_L + U * (chain * first + 4 * second + 4))
    if ids is None:
        assert logp is None
    else:
        t = want["ti"].abs()
        same_or_close(logp, want["logp"], tol_L + 4 * U * torch.where(torch.isfinite(t), t, 0.0))
    if top:
        assert torch.equal(top_ids.cpu(), want["top_ids"])
        d = want["top_logp"]
        same_or_close(top_logp, d, tol_L[:, None] + 4 * U * torch.where(torch.isfinite(d), d.abs() + want["stats"][:, 1:].nan_to_num().abs(), 0.0))
    else:
        assert top_ids is None and top_logp is None
    return got


def check_backward(mu, x, ids, scale, stats, H, dl, dh, dev=None, out=None):
    sc = float(torch.tensor(scale, dtype=F32))
    want, size = ref.logprobs_grad(x, ids, stats.cpu(), dl, sc, None if dh is None else H.cpu(), dh)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = mu.muon_token_logprobs_backward(x.cuda() if dev is None else dev, c(ids), stats, c(dl), scale=scale,
                                          entropy=None if dh is None else H, dentropy=c(dh), dlogits=out)
    assert got.dtype is x.dtype
    tiny = 2.0**-125   # what float32 leaves of a product near its smallest
    same_or_close(got, want, 32 * U * size + HALF[x.dtype] * (want.abs() + 32 * U * size) + tiny)
    return got


def make(kind, rows, vocab, dtype, gen):
    x = 3.0 * torch.randn(rows, vocab, generator=gen)
    if kind == "ties":
        x = torch.round(x / 2)
    elif kind == "equal":
        x = torch.full_like(x, -1.5)
    elif kind == "rising":
        x = torch.linspace(-20, 10, vocab).expand(rows, vocab).clone()
    elif kind == "falling":
        x = torch.linspace(10, -20, vocab).expand(rows, vocab).clone()
    elif kind == "masked":
        x[torch.rand(rows, vocab, generator=gen) < 0.7] = -math.inf
        x[0, :] = -math.inf
        if rows > 1:
            x[1, :] = -math.inf
            x[1, vocab // 2] = 4.0
    elif kind == "lowest":
        low = torch.finfo(dtype).min
        x[torch.rand(rows, vocab, generator=gen) < 0.5] = low
        x[0, :] = low
        if rows > 1:
            x[1, :] = -math.inf
            x[1, -1] = low
    elif kind == "huge":
        x = x * 1e37
    elif kind == "lost":
        x[0, vocab // 2] = math.nan
        x[-1, vocab // 3] = math.inf
    elif kind == "zeros":
        x = torch.where(torch.rand(rows, vocab, generator=gen) < 0.5, 0.0, -0.0)
    return x.to(dtype)


VOCABS = [1, 2, 7, 8, 9, 255, 256, 2047, 4097, 8191, 8193, 50280]
KINDS = ["plain", "ties", "equal", "rising", "falling", "masked", "lowest", "huge", "lost", "zeros"]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprobs(mu, vocab, kind, dtype):
    gen = torch.Generator().manual_seed(vocab)
    rows = 3 if vocab > 1000 else 9
    x = make(kind, rows, vocab, dtype, gen)
    ids = torch.randint(0, vocab, (rows,), generator=gen)
    ids[rows // 2] = -1
    if rows > 5:
        ids[5] = vocab
    for scale, top in ((1.0, 20), (0.75, 0), (1.25, 64), (1.0, 1)):
        if kind == "huge" and scale > 1.0:
            continue
        logp, H, stats, _, _ = check_forward(mu, x, ids, scale, top)
        dl, dh = torch.randn(rows, generator=gen), torch.randn(rows, generator=gen)
        if kind == "lost":   # those rows' gradients are NaN too, unless they take none
            dl[0] = 0.0
            dh[0] = 0.0
        check_backward(mu, x, ids, scale, stats, H, dl, dh)
        check_backward(mu, x, ids, scale, stats, H, dl, None)
    check_backward(mu, x, None, scale, stats, H, None, dh)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 64, 127, 128, 300, 511, 512, 700])
def test_rows_share_workgroups_or_not(mu, rows, dtype):
    gen = torch.Generator().manual_seed(rows)
    x, ids = make("ties", rows, 20011, dtype, gen), torch.randint(0, 20011, (rows,), generator=gen)
    check_forward(mu, x, ids, 1.0, 5)
    check_forward(mu, x, ids.int(), 1.0, 0)
    one = mu.muon_token_logprobs(x.cuda(), None, entropy=False, top=3)
    assert one[0] is None and one[1] is None
    assert torch.equal(one[3].cpu(), ref.logprobs(x, top=3)["top_ids"])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_strides_and_in_place(mu, dtype):
    """Columns of a padded tensor at an odd element, tokens a column, one gradient for all rows."""
    gen = torch.Generator().manual_seed(2)
    rows, vocab = 37, 10007
    x = make("masked", rows, vocab, dtype, gen)
    wide = torch.full((rows, vocab + 13), float("nan")).to(dtype)
    wide[:, 3:3 + vocab] = x
    w = wide.cuda()
    dev = w[:, 3:3 + vocab]
    text = torch.randint(-1, vocab, (rows, 4), generator=gen)
    logp, H, stats, _, _ = check_forward(mu, x, text[:, 1], 1.0, 7, dev=dev)
    again = mu.muon_token_logprobs(dev, text.cuda()[:, 1], top=7)
    assert torch.equal(again[0], logp) and torch.equal(again[1], H)
    dl, dh = torch.tensor([-0.25]).expand(rows), torch.randn(rows, generator=gen)
    sep = check_backward(mu, x, text[:, 1], 1.0, stats, H, dl, dh, dev=dev)
    one = mu.muon_token_logprobs_backward(dev, text.cuda()[:, 1], stats, torch.tensor([-0.25], device="cuda").expand(rows), entropy=H,
                                          dentropy=dh.cuda())
    assert torch.equal(one, sep)
    got = mu.muon_token_logprobs_backward(dev, text.cuda()[:, 1], stats, dl.cuda(), entropy=H, dentropy=dh.cuda(), dlogits=dev)
    assert got is dev and torch.equal(dev, sep)
    assert torch.isnan(w[:, :3]).all() and torch.isnan(w[:, 3 + vocab:]).all()


def test_leading_dimensions(mu):
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(2, 5, 300, generator=gen).cuda()
    text = torch.randint(0, 300, (2, 6), generator=gen).cuda()
    deep = mu.muon_token_logprobs(x, text[:, 1:], top=4)
    flat = mu.muon_token_logprobs(x.reshape(10, 300), text[:, 1:].reshape(10), top=4)
    assert [tuple(t.shape) for t in deep] == [(2, 5), (2, 5), (2, 5, 2), (2, 5, 4), (2, 5, 4)]
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(deep, flat))
    g = torch.full((1, 1), -0.1, device="cuda").expand(2, 5)
    assert torch.equal(mu.muon_token_logprobs_backward(x, text[:, 1:], deep[2], g).reshape(10, 300),
                       mu.muon_token_logprobs_backward(x.reshape(10, 300), text[:, 1:].reshape(10), flat[2], g.contiguous().reshape(10)))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_padding_rows_take_no_gradient(mu, dtype):
    """Whatever their logits hold."""
    x = torch.randn(4, 1000).to(dtype)
    x[1] = float("nan")
    x[2] = float("inf")
    x[3] = -math.inf
    ids = torch.tensor([5, -1, 1000, 7])
    logp, H, stats, _, _ = mu.muon_token_logprobs(x.cuda(), ids.cuda())
    assert logp[1] == 0 and logp[2] == 0 and logp[3] == -math.inf
    dx = mu.muon_token_logprobs_backward(x.cuda(), ids.cuda(), stats, torch.ones(4, device="cuda"))
    assert bool(dx[0].any()) and (dx[1:] == 0).all()


def test_probability_near_one(mu):
    """log p keeps its digits where the token takes nearly all: it is not a difference of two large numbers."""
    x = torch.zeros(3, 4096)
    x[:, 17] = torch.tensor([20.0, 30.0, 12.0]) + 100.0
    x += 64.0
    r = ref.logprobs(x, torch.tensor([17, 17, 17]))
    logp = mu.muon_token_logprobs(x.cuda(), torch.tensor([17, 17, 17]).cuda())[0]
    # the sum is 1 + 4095 e^-t: 2^-24 of it is all that is lost
    assert float((logp.double().cpu() - r["logp"]).abs().max()) <= 2 * U


def test_no_rows(mu):
    e = torch.empty(0, 50, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    logp, H, stats, top_ids, top_logp = mu.muon_token_logprobs(e, ids, top=3)
    assert logp.shape == (0,) and top_ids.shape == (0, 3)
    assert mu.muon_token_logprobs_backward(e, ids, stats, logp).shape == (0, 50)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 600])
def test_all_but_the_end_forbidden(mu, rows, dtype):
    """Nothing to set a bar by at first, then every logit better than all before it."""
    vocab, first = 40_011, 17_000
    x = torch.full((rows, vocab), -math.inf)
    x[:, first:] = torch.linspace(-30.0, 30.0, vocab - first)
    x = x.to(dtype)
    ids = torch.full((rows,), vocab - 5)
    check_forward(mu, x, ids, 1.0, 64)
    x[:, -40:] = -math.inf
    x[:, first:first + 30_000] = -math.inf
    check_forward(mu, x, ids, 1.0, 64)
