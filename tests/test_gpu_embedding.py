"""GPU parity of the token embedding and its gradient with the float64 reference
(tests/tok_reference.py).

Tolerances, element by element.  Forward: one product and one rounding to float32
(2^-24 each) and, for bfloat16, one to it (2^-8).  Gradient: a sum is a chain of at
most 64 additions in a chunk or two, then one of a sixteenth of the parts and 16
more, each off by 2^-24 of the sum of absolute values."""
import pytest

import tok_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0**-8, F32: 0.0}


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


def close(got, want, size, steps, dtype):
    """|got - want| within `steps` float32 roundings of size and one to dtype."""
    err = (got.double().cpu() - want).abs()
    bound = steps * 2.0**-24 * size + HALF[dtype] * (want.abs() + steps * 2.0**-24 * size) + 1e-44
    assert got.dtype is dtype and (err <= bound).all(), float((err - bound).max())


def grad_steps(tokens):
    return 64 + tokens // (16 * 16) + 16 + 4


def make_ids(kind, tokens, vocab, gen):
    if kind == "same":
        return torch.full((tokens,), vocab // 2)
    if kind == "sorted":
        return torch.sort(torch.randint(0, vocab, (tokens,), generator=gen)).values
    if kind == "often":      # shares of one over the rank, and padding
        rank = (torch.exp(torch.rand(tokens, generator=gen, dtype=torch.float64) * torch.tensor(float(vocab)).log()) - 1).long()
        ids = rank.clamp(0, vocab - 1) * 7919 % vocab
        return torch.where(torch.rand(tokens, generator=gen) < 0.1, torch.randint(-3, 0, (tokens,), generator=gen), ids)
    ids = torch.randint(-2, vocab + 2, (tokens,), generator=gen)     # outside on either side
    if tokens > 2:
        ids[0], ids[1] = -(2**62), 2**62
    return ids


@pytest.mark.parametrize("table", [BF16, F32], ids=["tbf16", "tf32"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens,vocab,n", [(1, 1, 1), (7, 10, 3), (33, 100, 4), (1000, 333, 5), (130, 50, 515), (64, 70, 768), (3, 9, 6000),
                                            (2500, 40, 96)])
def test_forward(mu, tokens, vocab, n, dtype, table):
    gen = torch.Generator().manual_seed(n)
    t = torch.randn(vocab, n, generator=gen).to(table)
    for kind in ("often", "outside"):
        ids = make_ids(kind, tokens, vocab, gen)
        for scale in (1.0, -27.7):
            want = ref.embedding(t, ids, float(torch.tensor(scale, dtype=F32)))
            got = mu.muon_embedding(t.cuda(), ids.cuda(), scale=scale, dtype=dtype)
            close(got, want, want.abs(), 2, dtype)
            if scale == 1.0 and dtype is table:
                assert torch.equal(got.double().cpu(), want)
    assert torch.equal(mu.muon_embedding(t.cuda(), ids.clamp(-9, 1 << 30).int().cuda(), scale=scale, dtype=dtype), got)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["often", "outside", "same", "sorted"])
@pytest.mark.parametrize("tokens,vocab,n", [(1, 1, 1), (15, 3, 5), (16, 2, 8), (17, 100, 515), (48, 2, 16), (64, 1, 768), (128, 9, 20), (129, 9, 20),
                                            (144, 2, 24), (1000, 257, 96),
                                            (3000, 5, 12), (5000, 70001, 8), (4097, 600, 33)])
def test_gradient(mu, tokens, vocab, n, kind, dtype):
    gen = torch.Generator().manual_seed(tokens + n)
    ids, dy = make_ids(kind, tokens, vocab, gen), torch.randn(tokens, n, generator=gen).to(dtype)
    want, size = ref.embedding_grad(dy, ids, vocab, 2.5)
    a = (dy.cuda(), ids.cuda(), vocab)
    got = mu.muon_embedding_backward(*a, scale=2.5)
    close(got, want, size, grad_steps(tokens), F32)
    close(mu.muon_embedding_backward(*a, scale=2.5, dtype=BF16), want, size, grad_steps(tokens), BF16)
    # again, with narrow ids, in a given tensor and workspace: the same bits
    out = torch.full((vocab, n), float("nan"), device="cuda")
    ws = torch.full((mu.muon_embedding_backward_workspace_size(ids, vocab, n),), 255, dtype=torch.uint8, device="cuda")
    r = mu.muon_embedding_backward(dy.cuda(), ids.clamp(-9, 1 << 30).int().cuda(), vocab, scale=2.5, dtable=out, workspace=ws)
    assert r is out and torch.equal(out, got)
    # added to what is there
    base = torch.randn(vocab, n, generator=gen)
    acc = base.cuda()
    mu.muon_embedding_backward(*a, scale=2.5, dtable=acc, accumulate=True)
    close(acc, base.double() + want, size + base.abs(), grad_steps(tokens) + 1, F32)
    untouched = torch.ones(vocab, dtype=torch.bool)
    untouched[ids[(ids >= 0) & (ids < vocab)]] = False
    assert torch.equal(acc.cpu()[untouched], base[untouched])


def test_runs_around_the_borders_of_chunks(mu):
    """Runs of every length from 1 to 70 behind one another, so that they start and end
    at every place of a chunk; and one that spans many."""
    gen = torch.Generator().manual_seed(3)
    counts = torch.cat([torch.arange(1, 71), torch.tensor([1, 900, 2]), torch.arange(70, 0, -1), torch.full((40,), 16), torch.full((20,), 32)])
    ids = torch.repeat_interleave(torch.arange(counts.numel()), counts)
    vocab = counts.numel() + 3
    for order in (torch.arange(ids.numel()), torch.randperm(ids.numel(), generator=gen)):
        for n in (8, 13):
            dy = torch.randn(ids.numel(), n, generator=gen)
            want, size = ref.embedding_grad(dy, ids[order], vocab)
            close(mu.muon_embedding_backward(dy.cuda(), ids[order].cuda(), vocab), want, size, grad_steps(ids.numel()), F32)


@pytest.mark.parametrize("kind", ["often", "same", "outside", "sorted"])
@pytest.mark.parametrize("tokens,vocab,n", [(40_960, 3, 8), (40_961, 100, 8), (41_000, 129, 5), (70_001, 66_000, 24), (131_071, 50_280, 3),
                                            (50_000, 600_000, 1)])
def test_many_tokens(mu, tokens, vocab, n, kind):
    """Around where ids are looked up before they are sorted, past where chunks are longer,
    ranges of one id and more ranges than are counted."""
    gen = torch.Generator().manual_seed(9)
    ids, dy = make_ids(kind, tokens, vocab, gen), torch.randn(tokens, n, generator=gen).to(BF16)
    want, size = ref.embedding_grad(dy, ids, vocab)
    a = (dy.cuda(), ids.cuda(), vocab)
    ws = torch.full((mu.muon_embedding_backward_workspace_size(ids, vocab, n),), 255, dtype=torch.uint8, device="cuda")
    got = mu.muon_embedding_backward(*a, workspace=ws)
    close(got, want, size, grad_steps(tokens), F32)
    assert torch.equal(got, mu.muon_embedding_backward(*a))
    # every other token of a wider tensor, narrow
    wide = torch.stack([ids, ids + 1], 1).clamp(-9, 1 << 30).int().cuda()
    assert torch.equal(got, mu.muon_embedding_backward(dy.cuda(), wide[:, 0], vocab))


def test_strides_and_odd_addresses(mu):
    gen = torch.Generator().manual_seed(4)
    text = torch.randint(-1, 60, (6, 41), generator=gen)
    wide = torch.randn(60, 131, generator=gen).to(BF16)
    table = wide.cuda()[:, 3:102]                    # rows 131 apart at an odd element
    buf = torch.full((6, 40, 120), float("nan"), device="cuda", dtype=BF16)
    for ids in (text[:, :-1], text[:, 1:], text.T[1:].T, text[:, ::3], text[2], text[:, 5], text[:1, :1].expand(4, 9)):
        want = ref.embedding(wide[:, 3:102], ids, 1.0)
        dev = text.cuda()
        view = dev.as_strided(ids.shape, ids.stride(), ids.storage_offset())
        got = mu.muon_embedding(table, view)
        assert torch.equal(got.double().cpu(), want)
        dy = torch.randn(*ids.shape, 99, generator=gen).to(BF16)
        grad = torch.zeros(*ids.shape, 107, dtype=BF16)
        grad[..., 5:104] = dy
        dwant, size = ref.embedding_grad(dy, ids, 60)
        close(mu.muon_embedding_backward(grad.cuda()[..., 5:104], view, 60), dwant, size, grad_steps(ids.numel()), F32)
    Y = buf[:, :, 7:106]
    assert mu.muon_embedding(table, text.cuda()[:, :-1], Y=Y) is Y
    assert torch.equal(Y.double().cpu(), ref.embedding(wide[:, 3:102], text[:, :-1]))
    assert torch.isnan(buf[:, :, :7]).all() and torch.isnan(buf[:, :, 106:]).all()


def test_padding_is_never_read(mu):
    """Rows of the gradient at padding hold anything; so do rows of the table that no token names."""
    gen = torch.Generator().manual_seed(5)
    ids = torch.tensor([3, -1, 0, 99, 3, 12])
    table = torch.randn(12, 16, generator=gen)
    table[[1, 2, 4, 5]] = float("nan")
    assert torch.equal(mu.muon_embedding(table.cuda(), ids.cuda()).double().cpu(), ref.embedding(table, ids))
    dy = torch.randn(6, 16, generator=gen)
    dy[[1, 3, 5]] = float("nan")
    want, size = ref.embedding_grad(torch.nan_to_num(dy), ids, 12)
    close(mu.muon_embedding_backward(dy.cuda(), ids.cuda(), 12), want, size, 8, F32)


@pytest.mark.parametrize("table", [BF16, F32], ids=["tbf16", "tf32"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [3, 128, 200, 1500])
def test_nothing_outside_the_table_is_written(mu, tokens, dtype, table):
    """Rows narrower than a piece, of a piece and a little wider, between guards."""
    gen = torch.Generator().manual_seed(tokens)
    for n in (1, 3, 4, 5, 6, 7, 8, 9, 15, 17, 130):
        vocab = 37
        ids, dy = make_ids("outside", tokens, vocab, gen), torch.randn(tokens, n, generator=gen).to(dtype)
        buf = torch.full(((vocab + 8) * n,), 3.0, dtype=table, device="cuda")
        out = buf[4 * n:-4 * n].view(vocab, n)
        mu.muon_embedding_backward(dy.cuda(), ids.cuda(), vocab, dtable=out)
        want, size = ref.embedding_grad(dy, ids, vocab)
        close(out, want, size, grad_steps(tokens), table)
        assert (buf[:4 * n] == 3.0).all() and (buf[-4 * n:] == 3.0).all(), n
        if table is F32:
            mu.muon_embedding_backward(dy.cuda(), ids.cuda(), vocab, dtable=out, accumulate=True)
            close(out, 2 * want, 2 * size, grad_steps(tokens) + 1, table)
            assert (buf[:4 * n] == 3.0).all() and (buf[-4 * n:] == 3.0).all(), n


def test_no_tokens(mu):
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    assert mu.muon_embedding(torch.randn(5, 8, device="cuda"), e).shape == (0, 8)
    got = mu.muon_embedding_backward(torch.empty(0, 8, device="cuda"), e, 5, dtable=torch.full((5, 8), 7.0, device="cuda"))
    assert (got == 0).all()
    got = mu.muon_embedding_backward(torch.empty(0, 8, device="cuda"), e, 5, dtable=torch.full((5, 8), 7.0, device="cuda"), accumulate=True)
    assert (got == 7.0).all()
    got = mu.muon_embedding_backward(torch.randn(4, 8, device="cuda"), torch.full((4,), -1, device="cuda"), 5)
    assert (got == 0).all()
