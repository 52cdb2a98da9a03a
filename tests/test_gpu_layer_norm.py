"""GPU parity of the layer norm and its gradients with the float64 reference
(tests/seq_reference.py).

Tolerances (relative 2-norm).  bfloat16 outputs are rounded once, 2^-9 at
most: 2e-3.  float32 outputs: sums of n (or rows) terms in trees of depth
about log n over partial sums of at most 64 terms, below 100 * 2^-24 = 6e-6:
1e-5."""
import pytest

import seq_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
TOL = {BF16: 2e-3, F32: 1e-5}


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


def inputs(rows, n, dtype, seed=0, affine=True):
    gen = torch.Generator().manual_seed(50 + seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (rn(rows, n) * (0.5 + torch.rand(n, generator=gen)) + 0.3).to(dtype)
    return x, (1.0 + 0.2 * rn(n) if affine else None), (0.1 * rn(n) if affine else None), rn(rows, n).to(dtype)


def cu(t):
    return None if t is None else t.cuda()


def check(mu, x, w, bias, dy, center, xg=None, dyg=None):
    xg = x.cuda() if xg is None else xg
    dyg = dy.cuda() if dyg is None else dyg
    y, mean, rstd = mu.muon_layer_norm(xg, cu(w), cu(bias), center=center)
    yr, mr, rr = ref.norm(x, w, bias, center=center)
    errs = {"y": (ref.rel(y, yr), TOL[x.dtype]), "rstd": (ref.rel(rstd, rr), 1e-5)}
    if center:
        errs["mean"] = (ref.rel(mean, mr), 1e-5)
    else:
        assert mean is None
    dx, dw, db = mu.muon_layer_norm_backward(dyg, xg, cu(w), mean, rstd, center=center, bias_grad=bias is not None)
    want = ref.norm_grads(dy, x, w, mean.cpu() if center else None, rstd.cpu(), center)
    errs["dx"] = (ref.rel(dx, want[0]), TOL[x.dtype])
    if w is not None:
        errs["dw"] = (ref.rel(dw, want[1]), 1e-5)
        errs["db"] = (ref.rel(db, want[2]), 1e-5)
    else:
        assert dw is None and db is None
    print("[parity] " + " ".join(f"{k} {v[0]:.2e}" for k, v in errs.items()), flush=True)
    assert all(a <= b for a, b in errs.values()), errs


# every layout of a row: one to four pieces a lane of a wave, of a workgroup, and longer; ragged ends of each
SIZES = [(7, 8), (5, 33), (130, 64), (33, 512), (9, 513), (64, 768), (11, 1500), (40, 2048), (5, 2049),
         (3, 4096), (17, 5000), (2, 8192), (3, 8200), (2, 20001), (700, 96)]


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,n", SIZES)
def test_norm(mu, rows, n, dtype, center):
    check(mu, *inputs(rows, n, dtype, seed=n), center)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,n", [(1, 1), (4, 1), (3, 2)])
def test_norm_one_or_two_elements(mu, rows, n, dtype, center):
    """Rows whose normalised elements are 0 or +-1 whatever they hold, so that
    dx is what its terms, of size r |t|, leave when they cancel: errors are
    taken relative to the terms, and a single element's rounding to bfloat16
    is 2^-8 of it (the 2e-3 of the larger cases is an average)."""
    x, w, bias, dy = inputs(rows, n, dtype, seed=n if n > 1 else 0)
    y, mean, rstd = mu.muon_layer_norm(x.cuda(), cu(w), cu(bias), center=center)
    yr, mr, rr = ref.norm(x, w, bias, center=center)
    assert ((y.cpu().double() - yr).abs() <= (2.0**-8 if dtype == BF16 else 1e-5) * yr.abs() + 1e-5).all()
    assert ref.rel(rstd, rr) <= 1e-5
    dx, dw, db = mu.muon_layer_norm_backward(dy.cuda(), x.cuda(), cu(w), mean, rstd, center=center)
    want = ref.norm_grads(dy, x, w, mean.cpu() if center else None, rstd.cpu(), center)
    terms = rstd.cpu().double()[:, None] * (dy.double() * w.double()).abs().sum(1, keepdim=True)
    assert ((dx.cpu().double() - want[0]).abs() <= (2.0**-8 if dtype == BF16 else 0.0) * want[0].abs() + 1e-5 * terms).all()
    if center and n == 1:
        assert torch.count_nonzero(dx) == 0 and torch.count_nonzero(dw) == 0
    else:
        assert ref.rel(dw, want[1]) <= 1e-5
    assert ref.rel(db, want[2]) <= 1e-5


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [255, 257, 511, 513, 1023, 1025, 2047, 2049, 4095, 4097, 8191, 8193, 16383, 16385])
def test_norm_lengths(mu, n, dtype):
    """Around the lengths where rows take another share of threads; rows that
    end inside a piece of 16 bytes."""
    check(mu, *inputs(9, n, dtype, seed=n), True)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 4, 5, 7, 8, 9])
def test_norm_short_rows(mu, n, dtype):
    """Rows of about one piece of 16 bytes: few elements, so by element."""
    test_norm_one_or_two_elements(mu, 9, n, dtype, True)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_norm_without_parameters(mu, dtype):
    check(mu, *inputs(50, 300, dtype, affine=False), True)


@pytest.mark.parametrize("rows", [31, 33, 5000, 20000])
def test_norm_many_rows(mu, rows):
    """One workgroup's rows and many: the column sums join in fixed order."""
    x, w, bias, dy = inputs(rows, 72, BF16, seed=rows)
    check(mu, x, w, bias, dy, True)
    a = mu.muon_layer_norm(x.cuda(), cu(w), cu(bias))
    r = [mu.muon_layer_norm_backward(dy.cuda(), x.cuda(), cu(w), a[1], a[2]) for _ in range(2)]
    assert all(torch.equal(i, j) for i, j in zip(*r))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off,ld", [(0, 776), (1, 800), (3, 771)])
def test_norm_strided_rows(mu, off, ld, dtype):
    """Rows inside a wider tensor, aligned for vector loads or not."""
    x, w, bias, dy = inputs(20, 768, dtype, seed=off)
    wide = torch.zeros(2, 20, ld + off, dtype=dtype, device="cuda")
    xg, dyg = wide[0, :, off:off + 768], wide[1, :, off:off + 768]
    xg.copy_(x)
    dyg.copy_(dy)
    check(mu, x, w, bias, dy, True, xg, dyg)


def test_norm_large_mean(mu):
    """A mean 1000 times the spread: the variance is taken around the mean.
    x is exact in float32, so only the statistics' own rounding counts: the
    mean's, 2^-24 * 1000 of the spread or 6e-5, is in y once."""
    gen = torch.Generator().manual_seed(3)
    x = (1000.0 + torch.randn(30, 1000, generator=gen)).float()
    y, mean, rstd = mu.muon_layer_norm(x.cuda())
    yr, mr, rr = ref.norm(x)
    assert ref.rel(y, yr) <= 2e-4 and ref.rel(mean, mr) <= 1e-6 and ref.rel(rstd, rr) <= 1e-5


def test_norm_constant_and_nonfinite_rows(mu):
    """A constant row gives the bias and finite gradients; a row with a NaN or
    an infinity is NaN and leaves the other rows alone."""
    x, w, bias, dy = inputs(6, 100, F32)
    x[1] = 4.0
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    y, mean, rstd = mu.muon_layer_norm(x.cuda(), cu(w), cu(bias))
    yr = ref.norm(x, w, bias)[0]
    assert torch.equal(y[1].cpu(), bias)
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).any()
    for i in (0, 1, 2, 5):
        assert ref.rel(y[i], yr[i]) <= 1e-5
    dx = mu.muon_layer_norm_backward(dy.cuda(), x.cuda(), cu(w), mean, rstd)[0]
    assert torch.isfinite(dx[[0, 1, 2, 5]]).all()


def test_norm_higher_dimensions_and_empty(mu):
    x, w, bias, dy = inputs(24, 40, F32)
    y, mean, rstd = mu.muon_layer_norm(x.cuda().view(2, 3, 4, 40), cu(w), cu(bias))
    assert y.shape == (2, 3, 4, 40) and mean.shape == (2, 3, 4)
    assert ref.rel(y.view(24, 40), ref.norm(x, w, bias)[0]) <= 1e-5
    e = torch.empty(0, 40, device="cuda")
    y, mean, rstd = mu.muon_layer_norm(e, cu(w), cu(bias))
    assert y.shape == (0, 40)
    for n in (40, 9000):
        e = torch.empty(0, n, device="cuda")
        dx, dw, db = mu.muon_layer_norm_backward(e, e, torch.ones(n, device="cuda"), e[:, 0].contiguous(), e[:, 0].contiguous())
        torch.cuda.synchronize()
        assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_norm_gradients_are_differences(mu):
    """float32 gradients against central differences of the float64 reference."""
    x, w, bias, dy = inputs(12, 50, F32, seed=9)
    for center in (True, False):
        _, mean, rstd = mu.muon_layer_norm(x.cuda(), cu(w), cu(bias), center=center)
        grads = mu.muon_layer_norm_backward(dy.cuda(), x.cuda(), cu(w), mean, rstd, center=center)
        gen = torch.Generator().manual_seed(7)
        args = [x.double(), w.double(), bias.double()]
        for i, g in enumerate(grads):
            d = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
            at = lambda s: float((ref.norm(*[a + s * d if j == i else a for j, a in enumerate(args)], center=center)[0]  # noqa: E731
                                  * dy.double()).sum())
            diff = (at(1e-5) - at(-1e-5)) / 2e-5
            g = g.cpu().double()
            assert abs(float((g * d).sum()) - diff) <= 1e-5 * float(g.norm() * d.norm())
