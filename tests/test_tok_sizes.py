"""Where the token operators' plans change with size, seen from the host (no GPU
needed: nothing is enqueued)."""
import pytest

from test_tok_abi import mu  # noqa: F401

torch = pytest.importorskip("torch")


def up(x):
    return (x + 255) // 256 * 256


def embedding_workspace(tokens, n, ranges):
    """Bytes of the sorted tokens and the part sums, and with `ranges` of the map of the tokens'
    ranges (16 bits each for sixteen waves, an odd number of 512 tokens to a wave) and its counts."""
    chunk = 32 if tokens > 1 << 16 else 16
    need = 256 + up(tokens * 8) + up((tokens + chunk - 1) // chunk * 2 * n * 4)
    if ranges:
        wave = (tokens + 15) // 16
        padded = 16 * (((wave + 511) // 512) | 1) * 512
        need += up(padded * 2) + up(padded // 2048 * ranges * 4)
    return need


@pytest.mark.parametrize("tokens,mapped", [(40_960, False), (40_961, True), (131_071, True), (134_209_536, True), (134_209_537, False),
                                           (134_217_727, False), (134_217_728, False), (134_217_729, False), (1 << 30, False)])
@pytest.mark.parametrize("vocab,ranges", [(100, 100), (50_280, 128)])
def test_the_map_of_ranges_holds_its_offsets(mu, tokens, mapped, vocab, ranges):  # noqa: F811
    """A token is listed as its place among its wave's, in the 23 bits beside those of its id: where a
    wave walks more than 2^23 tokens, ranges are not looked up first."""
    wave = (tokens + 15) // 16
    assert not mapped or (((wave + 511) // 512) | 1) * 512 <= 1 << 23
    got = mu.lib().muon_embedding_backward_workspace_size(tokens, vocab, 1)
    assert got == embedding_workspace(tokens, 1, ranges if mapped else 0)


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, 1), (torch.float32, 0)])
@pytest.mark.parametrize("shape,groups", [((700, 192), 3), ((2, 5, 96), 1), ((96,), 4), ((0, 96), 2), ((16_384, 1536), 1), ((4, 40_002), 1),
                                          ((2062, 24 * 75), 24)])
def test_group_norm_backward_workspace(mu, shape, groups, dtype, code):  # noqa: F811
    """The binding's size is the library's: that of the parts of two sums at least."""
    X = torch.empty(shape, dtype=dtype)
    rows, n = X.numel() // shape[-1], shape[-1]
    got = mu.muon_group_norm_backward_workspace_size(X, groups)
    assert got == mu.lib().muon_group_norm_backward_workspace_size(rows, groups, n // groups, code) >= 2 * n * 4


@pytest.mark.parametrize("call,error", [
    (lambda m: m.muon_group_norm_backward_workspace_size(torch.empty(3, 8), 3), ValueError),
    (lambda m: m.muon_group_norm_backward_workspace_size(torch.empty(3, 8), 0), ValueError),
    (lambda m: m.muon_group_norm_backward_workspace_size(torch.empty(3, 8).half(), 2), TypeError),
    (lambda m: m.muon_group_norm_backward_workspace_size(torch.empty(0, 1 << 32), 1), RuntimeError),
])
def test_group_norm_backward_workspace_refusals(mu, call, error):  # noqa: F811
    with pytest.raises(error):
        call(mu)


@pytest.mark.parametrize("scale,status", [(3e38, -1), (2.36e38, -1), (2.35e38, 0), (1e-45, 0)])
def test_largest_scale(mu, scale, status):  # noqa: F811
    """Exponents are taken in base 2: past the largest float32 over log2(e) the factor was an infinity, and
    0 times it, at the largest logit, NaN."""
    from test_tok_abi import logp, logp_bwd
    assert logp(mu, rows=0, scale=scale) == status and logp_bwd(mu, rows=0, scale=scale) == status
