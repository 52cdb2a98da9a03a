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
