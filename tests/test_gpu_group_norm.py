"""GPU parity of the group norm and its gradients with the float64 reference
(tests/tok_reference.py).

Tolerances, element by element: what float32 leaves, as group_norm_bounds derives
it, and for bfloat16 results one rounding more, half a step of 2^-8 at most.  The
statistics: 100 roundings of 2^-24 and those of their inputs, 1e-5."""
import pytest

import tok_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0**-8, F32: 0.0}
MODES = {"before": (True, True, "silu"), "after": (True, False, "silu"), "silu": (False, True, "silu"), "none": (False, True, "none")}


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


def rel(got, want):
    return float((got.double().cpu() - want).norm() / want.norm().clamp_min(1e-30))


def cu(t):
    return None if t is None else t.cuda()


def inputs(rows, n, dtype, seed=0, affine=True, gated=True):
    gen = torch.Generator().manual_seed(60 + seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=(rn(rows, n) * (0.5 + torch.rand(n, generator=gen)) + 0.3).to(dtype), z=(2.0 * rn(rows, n)).to(dtype) if gated else None,
                w=1.0 + 0.2 * rn(n) if affine else None, b=0.1 * rn(n) if affine else None, dy=rn(rows, n).to(dtype))


def check(mu, i, groups, mode, center, dev=None):
    """dev: the operands on the GPU where they are not plain copies."""
    gated, first, act = MODES[mode]
    x, z, w, b, dy = (i[k] for k in ("x", "z", "w", "b", "dy"))
    g = {k: cu(v) for k, v in i.items()}
    g.update(dev or {})
    kw = dict(gate=g["z"], gate_first=first, activation=act, center=center)
    y, mean, rstd = mu.muon_group_norm(g["x"], groups, g["w"], g["b"], **kw)
    yr, mr, rr = ref.group_norm(x, groups, w, b, z, first, act, 1e-5, center)
    far = {"rstd": rel(rstd, rr) / 1e-5}
    assert y.dtype is x.dtype and (mean is not None) == center
    if center:
        size = float(torch.linalg.vector_norm(mr)) + 1e-2 * mr.numel() ** 0.5   # (a mean near 0 is off by its terms' roundings)
        far["mean"] = float((mean.double().cpu() - mr).norm()) / size / 1e-5
    bounds = ref.group_norm_bounds(dy, x, groups, w, b, mr, rr, z, first, act, forward=True)
    dx, dz, dw, db = mu.muon_group_norm_backward(g["dy"], g["x"], groups, g["w"], g["b"], mean, rstd, **kw)
    stats = cu_back(mean), cu_back(rstd)
    want = ref.group_norm_grads(dy, x, groups, w, b, *stats, z, first, act)
    bounds.update(ref.group_norm_bounds(dy, x, groups, w, b, *stats, z, first, act))
    assert (dz is not None) == gated and (dw is not None) == (w is not None) and (db is not None) == (b is not None)
    for name, got, v in zip(("y", "dx", "dz", "dw", "db"), (y, dx, dz, dw, db), (yr, *want)):
        if got is None:
            continue
        half = HALF[x.dtype] if name in ("y", "dx", "dz") else 0.0
        e = bounds[name] + half * (v.abs() + bounds[name]) + 1e-37
        far[name] = float(((got.double().cpu() - v).abs() / e).max())
    print("[parity] of the bounds: " + " ".join(f"{k} {v:.3f}" for k, v in far.items()), flush=True)
    assert all(v <= 1 for v in far.values()), far
    return y, dx


def cu_back(t):
    return None if t is None else t.cpu()


# every layout of a group: under a piece, 8 and 16 threads, one to four pieces of a wave, workgroups, and longer
SIZES = [(7, 1, 1), (50, 40, 3), (5, 3, 8), (1, 1, 33), (33, 24, 64), (130, 24, 75), (9, 2, 100), (17, 3, 128), (12, 1, 200), (40, 2, 256),
         (6, 1, 513), (11, 2, 768), (300, 1, 1024), (64, 1, 1536), (5, 1, 2048), (3, 2, 2049), (4, 1, 4000), (3, 1, 8191), (2, 1, 12001),
         (2, 1, 20001), (700, 1, 96)]


@pytest.mark.parametrize("center", [True, False], ids=["center", "rms"])
@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,groups,width", SIZES)
def test_group_norm(mu, rows, groups, width, dtype, mode, center):
    check(mu, inputs(rows, groups * width, dtype, seed=width, affine=(rows + width) % 3 != 0, gated=MODES[mode][0]), groups, mode, center)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mode", list(MODES))
def test_slices_of_a_projection(mu, mode, dtype):
    """x and z are column ranges of one tensor, at odd elements."""
    i = inputs(37, 6 * 44, dtype, gated=MODES[mode][0])
    n = 6 * 44
    wide = torch.full((37, 2 * n + 31), float("nan")).to(dtype)
    wide[:, 5:5 + n] = i["x"]
    dev = {}
    if i["z"] is not None:
        wide[:, n + 12:2 * n + 12] = i["z"]
    w = wide.cuda()
    dev["x"] = w[:, 5:5 + n]
    if i["z"] is not None:
        dev["z"] = w[:, n + 12:2 * n + 12]
    check(mu, i, 6, mode, True, dev)
    out = torch.full((37, n + 9), float("nan"), dtype=dtype, device="cuda")
    kw = dict(gate=dev.get("z"), gate_first=MODES[mode][1], activation=MODES[mode][2])
    Y = out[:, 3:3 + n]
    want = mu.muon_group_norm(dev["x"], 6, cu(i["w"]), **kw)[0]
    assert mu.muon_group_norm(dev["x"], 6, cu(i["w"]), Y=Y, **kw)[0] is Y and torch.equal(Y, want)
    assert torch.isnan(out[:, :3]).all() and torch.isnan(out[:, 3 + n:]).all()


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("width", [4, 64, 300, 3000])
def test_a_group_is_by_itself(mu, width, mode):
    """What is not finite in one group of one row stays there."""
    gated, first, act = MODES[mode]
    i = {k: cu(v) for k, v in inputs(6, 4 * width, F32, gated=gated).items()}
    i["b"] = None
    kw = dict(gate=i["z"], gate_first=first, activation=act)
    bad = {k: v.clone() if v is not None else None for k, v in i.items()}
    bad["x"][2, width + width // 2] = float("nan")
    bad["x"][4, 3 * width] = float("inf")
    hit = torch.zeros(6, 4, dtype=torch.bool)
    hit[2, 1] = hit[4, 3] = True
    y, _, rstd = mu.muon_group_norm(i["x"], 4, i["w"], **kw)
    yb, _, rb = mu.muon_group_norm(bad["x"], 4, i["w"], **kw)
    same = lambda a, b: (a.unflatten(1, (4, -1)) == b.unflatten(1, (4, -1))).all(2).cpu()  # noqa: E731
    assert same(y, yb)[~hit].all() and not same(y, yb)[hit].any()
    dx = mu.muon_group_norm_backward(i["dy"], i["x"], 4, i["w"], None, None, rstd, **kw)[0]
    db = mu.muon_group_norm_backward(i["dy"], bad["x"], 4, i["w"], None, None, rb, **kw)[0]
    assert same(dx, db)[~hit].all() and not same(dx, db)[hit].any()


def test_far_gates(mu):
    """silu and its slope where e^-z leaves float32: 0 and z, 0 and 1."""
    z = torch.tensor([-200.0, -100.0, -89.0, -30.0, 0.0, 30.0, 89.0, 100.0, 200.0, 3e38, -3e38, 1.0]).repeat(5, 4)
    gen = torch.Generator().manual_seed(8)
    x, dy = torch.randn(5, 48, generator=gen), torch.randn(5, 48, generator=gen)
    y, _, rstd = mu.muon_group_norm(x.cuda(), 1, gate=z.cuda(), gate_first=False)
    yr, _, rr = ref.group_norm(x, 1, z=z, gate_first=False)
    # (3e38 times a norm above 1.13 lies past float32: its rounding is an infinity, which allclose wants equal)
    assert torch.allclose(y.cpu(), yr.float(), rtol=1e-5, atol=1e-30)
    dx, dz, _, _ = mu.muon_group_norm_backward(dy.cuda(), x.cuda(), 1, None, None, None, rstd, gate=z.cuda(), gate_first=False)
    assert torch.isfinite(dz).all()
    keep = z.abs() < 1e30
    want = ref.group_norm_grads(torch.where(keep, dy, 0.0), x, 1, None, None, None, rstd.cpu(), torch.where(keep, z, 0.0), False)[1]
    assert torch.allclose(torch.where(keep, dz.double().cpu(), 0.0), want, rtol=1e-4, atol=1e-25)


def test_large_mean(mu):
    """The variance is taken around the mean."""
    gen = torch.Generator().manual_seed(3)
    x = (1000.0 + torch.randn(30, 1000, generator=gen)).float()
    y, mean, rstd = mu.muon_group_norm(x.cuda(), 4, center=True, activation="none")
    yr, mr, rr = ref.group_norm(x, 4, activation="none", center=True)
    # the mean is off by 2^-24 of 1000 or two, which moves every result by as much
    assert rel(rstd, rr) < 1e-5 and float((y.double().cpu() - yr).abs().max()) < 4 * 1000 * 2.0**-24


@pytest.mark.parametrize("rows", [0, 1])
@pytest.mark.parametrize("groups", [1, 3])
def test_few_rows(mu, rows, groups):
    x, z, w = torch.randn(rows, 96, device="cuda"), torch.randn(rows, 96, device="cuda"), torch.randn(96, device="cuda")
    y, mean, rstd = mu.muon_group_norm(x, groups, w, w, gate=z, center=True)
    assert y.shape == (rows, 96) and mean.shape == rstd.shape == (rows, groups)
    dx, dz, dw, db = mu.muon_group_norm_backward(x, x, groups, w, w, mean, rstd, gate=z, center=True)
    assert dx.shape == dz.shape == (rows, 96)
    if rows == 0:
        assert (dw == 0).all() and (db == 0).all()


def test_many_rows(mu):
    """More workgroups than one dimension of a grid takes here, and sums over many rows."""
    rows = (1 << 20) * 32 + 77
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(rows, 8, generator=gen, device="cuda").to(BF16)
    y, _, rstd = mu.muon_group_norm(x, 1, activation="none")
    xd = x[-1000:].double()
    want = xd / torch.sqrt(xd.square().mean(1, keepdim=True) + 1e-5)
    assert rel(y[-1000:], want.cpu()) < 2.0**-8 + 1e-5
    assert bool((rstd > 0).all())


def test_leading_dimensions(mu):
    i = inputs(24, 128, BF16)
    args = lambda s: (i["x"].cuda().reshape(s), 2, i["w"].cuda())  # noqa: E731
    z = i["z"].cuda()
    flat = mu.muon_group_norm(*args((24, 128)), gate=z, center=True)
    deep = mu.muon_group_norm(*args((2, 3, 4, 128)), gate=z.reshape(2, 3, 4, 128), center=True)
    assert deep[0].shape == (2, 3, 4, 128) and deep[1].shape == deep[2].shape == (2, 3, 4, 2)
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(deep, flat))


@pytest.mark.parametrize("dtype,width", [(BF16, 1200), (F32, 700)], ids=["bf16", "f32"])
@pytest.mark.parametrize("mode", list(MODES))
def test_more_rows_than_workgroups_take_at_once(mu, mode, dtype, width):
    """Three pieces a thread, whose workgroups are fewer with a gate."""
    check(mu, inputs(17_000, width, dtype, seed=2, gated=MODES[mode][0]), 1, mode, True)


@pytest.mark.parametrize("rows,groups,width", [(3, 5000, 1), (300, 700, 3), (2, 1500, 9), (1, 600, 70)])
def test_many_groups(mu, rows, groups, width):
    check(mu, inputs(rows, groups * width, F32, seed=4), groups, "before", True)


@pytest.mark.parametrize("rows,groups,width", [(5, 3, 40), (1500, 2, 300), (700, 1, 9000)])
def test_one_parameter(mu, rows, groups, width):
    """A weight or a bias alone: its gradient, and the others', as with both where the other is 1 or 0."""
    i = {k: cu(v) for k, v in inputs(rows, groups * width, BF16).items()}
    one, zero = torch.ones_like(i["w"]), torch.zeros_like(i["w"])
    for center in (True, False):
        def both(w, b):
            y, mean, rstd = mu.muon_group_norm(i["x"], groups, w, b, gate=i["z"], gate_first=False, center=center)
            return y, *mu.muon_group_norm_backward(i["dy"], i["x"], groups, w, b, mean, rstd, gate=i["z"], gate_first=False, center=center)
        for (w, b), (w2, b2) in (((i["w"], None), (i["w"], zero)), ((None, i["b"]), (one, i["b"])), ((None, None), (one, zero))):
            got, want = both(w, b), both(w2, b2)
            assert (got[3] is None) == (w is None) and (got[4] is None) == (b is None)
            assert all(g is None or torch.equal(g, v) for g, v in zip(got, want))
