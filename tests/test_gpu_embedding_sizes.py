"""The embedding's gradient at its largest numbers of tokens, exactly: gradients of 1
and -1 at random, whose sums in any order are whole numbers far below 2^24 (the
square root of 2^30 tokens is 2^15)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


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


def signs(tokens, vocab, seed):
    """(dy [tokens, 1], ids with some padding, the sums [vocab, 1])."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.empty(tokens, dtype=torch.int32, device="cuda").random_(-1, vocab, generator=gen)
    dy = torch.empty(tokens, 1, dtype=BF16, device="cuda").random_(0, 2, generator=gen).mul_(2).sub_(1)
    want = torch.zeros(vocab + 1, dtype=torch.float64, device="cuda")
    for a in range(0, tokens, 1 << 24):
        part = slice(a, a + (1 << 24))
        want += torch.bincount(ids[part] + 1, weights=dy[part, 0].double(), minlength=vocab + 1)
    return dy, ids, want[1:, None].float()


@pytest.mark.parametrize("tokens", [134_209_536, 134_209_537, (1 << 27) - 1, 1 << 27])
def test_where_the_map_of_ranges_ends(mu, tokens):
    """Up to 2^23 tokens a wave ranges are looked up first; past that a place among a wave's
    tokens no longer fits beside an id."""
    dy, ids, want = signs(tokens, 100, seed=tokens & 7)
    assert torch.equal(mu.muon_embedding_backward(dy, ids, 100), want)


@pytest.mark.parametrize("tokens,vocab", [(1 << 30, 3), (1 << 30, 100)])
def test_most_tokens(mu, tokens, vocab):
    """Runs of so many chunks that four of them to a workgroup are 2^32 work items."""
    dy, ids, want = signs(tokens, vocab, seed=vocab)
    assert torch.equal(mu.muon_embedding_backward(dy, ids, vocab), want)


def additions(tokens):
    """The longest chain of additions to an element: two chunks of sorted tokens, then of the chunks'
    parts those of one wave in eight, the eight waves' sums and what was there; and the scale (more than 128 tokens)."""
    chunk = 32 if tokens > 1 << 16 else 16
    return 2 * chunk + -(-(-(-tokens // chunk)) // 8) + 8 + 2


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [257, 515, 1030])
@pytest.mark.parametrize("tokens", [1000, 50_000, 70_000])
def test_long_runs_of_wide_rows(mu, tokens, n, dtype):
    """Parts of several slices of a row's columns, within additions() roundings of 2^-24 of the sum
    of absolute values: one id, and ids with runs across a few borders."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    dy = torch.rand(tokens, n, generator=gen, device="cuda").add_(0.5).to(dtype)
    one = torch.full((tokens,), 2, device="cuda")
    some = torch.randint(-1, tokens // 100, (tokens,), generator=gen, device="cuda")
    for ids, vocab in ((one, 5), (some, tokens // 100)):
        want = torch.zeros(vocab + 1, n, dtype=torch.float64, device="cuda").index_add_(0, ids + 1, dy.double())[1:] * 0.75
        for accumulate in (False, True):
            got = torch.ones(vocab, n, device="cuda")
            mu.muon_embedding_backward(dy, ids, vocab, scale=0.75, dtable=got, accumulate=accumulate)
            sums = want + 1 if accumulate else want
            assert ((got.double() - sums).abs() <= additions(tokens) * 2.0**-24 * sums).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [6, 129, 500, 41_000])
def test_padding_holds_anything(mu, tokens, dtype):
    """Rows at padding, the first among them, are NaN, and so are those of ids past the table; the
    tokens that count do not fill their last chunk.  (Up to 128 tokens one chain may add them all.)"""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    ids = torch.randint(-3, 40, (tokens,), generator=gen, device="cuda")
    ids[0], ids[-1] = -1, 31
    for vocab, n in ((31, 20), (40, 1), (1000, 300)):
        dy = torch.randn(tokens, n, generator=gen, device="cuda").to(dtype)
        there = (ids >= 0) & (ids < vocab)
        dy[~there] = float("nan")
        want, size = (torch.zeros(vocab, n, dtype=torch.float64, device="cuda").index_add_(0, ids[there], v) for v in
                      (dy[there].double(), dy[there].double().abs()))
        got = mu.muon_embedding_backward(dy, ids, vocab)
        assert ((got.double() - want).abs() <= (additions(tokens) + 128) * 2.0**-24 * size).all()
