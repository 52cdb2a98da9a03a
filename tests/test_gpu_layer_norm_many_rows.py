"""Layer norm of more rows than a launch has work items for in one dimension
(2^32): the rows past that are computed like the others, bit for bit what
calls on parts of them give."""
import pytest

import seq_reference as ref
from test_gpu_layer_norm import BF16, TOL, _announce, mu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PART = 1 << 16


@pytest.mark.parametrize("rows,n", [((1 << 24) + 77, 4),     # rows shorter than 16 bytes: a workgroup each
                                    ((1 << 26) + 5, 8),      # four rows a workgroup
                                    ((1 << 24) + 3, 2056)])  # a workgroup each
def test_many_rows(mu, rows, n):
    gen = torch.Generator(device="cuda").manual_seed(61)
    # the rows repeat after a while: inputs are made quickly, and parts far apart can be told from each other
    some = torch.randn(9973, n, generator=gen, device="cuda").to(BF16)
    x = torch.empty(rows, n, dtype=BF16, device="cuda")
    for at in range(0, rows, 1 << 22):
        hi = min(rows, at + (1 << 22))
        x[at:hi] = some[torch.arange(at, hi, device="cuda") % 9973]
    w = 1.0 + 0.1 * torch.randn(n, generator=gen, device="cuda")
    y, mean, rstd = mu.muon_layer_norm(x, w)
    for at in (0, PART, rows // 2, (1 << 24) - 3, rows - PART):
        part = slice(at, min(rows, at + PART))
        a, b, c = mu.muon_layer_norm(x[part], w)
        assert torch.equal(y[part], a) and torch.equal(mean[part], b) and torch.equal(rstd[part], c)
    want = ref.norm(x[-PART:].cpu(), w.cpu())[0]
    assert ref.rel(y[-PART:], want) <= TOL[BF16]
