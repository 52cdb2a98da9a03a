"""GPU parity of the gated scan, its gradients and its single-token form with
the float64 reference (tests/seq_reference.py).

Tolerances (relative 2-norm).  bfloat16 outputs: a value passes at most three
roundings to bfloat16 (a product's weights or the state copy it reads, a sum's
operand, the result), each at most 2^-8 relative and 1.7e-3 in the mean
square; three independent ones leave 2.9e-3, and twice that is allowed: 6e-3.  float32
outputs (states, gate gradients, everything with float32 inputs): the
operands keep 24 bits and the sums have at most a few hundred terms at a time;
random rounding of n terms leaves sqrt(n) 2^-24 ~ 2e-6, and the chunks' decays
add a few units more: 1e-5, the bound of the other float32 paths."""
import math

import pytest

import seq_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16_TOL = 6e-3
F32_TOL = 1e-5


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


def inputs(B, T, H, G, P, N, dtype, seed=0, gate=True, state=True, resets=0.0, decay=0.1, sliced=False):
    """Seeded inputs on the CPU: normal v, k, q, dy, states; log decays
    -decay * |normal| with a share of resets; gates in [0, 1)."""
    gen = torch.Generator().manual_seed(1000 + seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = {}
    if sliced:   # column ranges of a wider tensor, rows that no vector load fits when the sizes are odd
        wide = rn(B, T, 3 + H * P + 2 * G * N).to(dtype)
        v, k, q = wide[..., 3:].split([H * P, G * N, G * N], dim=2)
    else:
        v, k, q = (rn(B, T, c).to(dtype) for c in (H * P, G * N, G * N))
    x["v"], x["k"], x["q"] = v.unflatten(2, (H, P)), k.unflatten(2, (G, N)), q.unflatten(2, (G, N))
    g = -decay * rn(B, T, H).abs()
    x["g"] = torch.where(torch.rand(B, T, H, generator=gen) < resets, -math.inf, g)
    x["b"] = torch.rand(B, T, H, generator=gen) if gate else None
    x["S0"] = rn(B, H, P, N) if state else None
    x["dy"] = rn(B, T, H, P).to(dtype)
    x["dS"] = rn(B, H, P, N) if state else None
    return x


def forward(mu, x, **kw):
    c = {n: None if t is None else t.cuda() for n, t in x.items()}
    return mu.muon_gated_scan(c["v"], c["k"], c["q"], c["g"], gate=c["b"], S0=c["S0"], **kw)


def backward(mu, x, **kw):
    c = {n: None if t is None else t.cuda() for n, t in x.items()}
    return mu.muon_gated_scan_backward(c["v"], c["k"], c["q"], c["g"], c["dy"], gate=c["b"], S0=c["S0"], dS=c["dS"], **kw)


def check_forward(mu, x):
    tol = BF16_TOL if x["v"].dtype == torch.bfloat16 else F32_TOL
    y, S = forward(mu, x)
    yr, Sr, _ = ref.scan(x["v"], x["k"], x["q"], x["g"], x["b"], x["S0"])
    e = (ref.rel(y, yr), ref.rel(S, Sr))
    print(f"[parity] y {e[0]:.2e} S {e[1]:.2e}", flush=True)
    assert y.dtype == x["v"].dtype and S.dtype == torch.float32
    assert e[0] <= tol and e[1] <= F32_TOL, e


def check_backward(mu, x):
    tol = BF16_TOL if x["v"].dtype == torch.bfloat16 else F32_TOL
    got = backward(mu, x)
    want = ref.scan_grads(x["v"], x["k"], x["q"], x["g"], x["dy"], x["b"], x["S0"], x["dS"])
    errs = {}
    for name, t, a, w in zip(("dv", "dk", "dq", "dg", "db", "dS0"), (tol, tol, tol, F32_TOL, F32_TOL, F32_TOL), got, want):
        if a is None:
            assert x["b" if name == "db" else "S0"] is None
            continue
        errs[name] = ref.rel(a, w)
        assert errs[name] <= t, errs
    print("[parity] " + " ".join(f"{n} {e:.2e}" for n, e in errs.items()), flush=True)


BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [  # B, T, H, G, P, N
    (1, 1, 1, 1, 1, 1),
    (2, 1, 4, 2, 64, 128),
    (1, 63, 2, 1, 64, 64),
    (1, 64, 2, 2, 32, 16),
    (2, 65, 3, 1, 40, 72),
    (1, 130, 4, 2, 64, 128),
    (3, 200, 2, 1, 17, 5),
    (1, 193, 2, 1, 130, 100),     # three blocks of value rows, the last of two
    (2, 300, 6, 3, 80, 128),
    (1, 1100, 1, 1, 64, 128),     # several segments of the time axis
    (1, 70, 24, 1, 64, 128),      # 24 heads on one group, split over workgroups
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_scan(mu, shape, dtype):
    check_forward(mu, inputs(*shape, dtype, seed=shape[1]))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_scan_backward(mu, shape, dtype):
    check_backward(mu, inputs(*shape, dtype, seed=shape[1]))


@pytest.mark.parametrize("shape", [(2, 1, 4, 2, 64, 128), (2, 2, 4, 2, 64, 64), (3, 2, 2, 1, 80, 128), (2, 17, 3, 1, 40, 72),
                                   (1, 64, 4, 2, 64, 128)], ids=str)
def test_short_bf16_is_rounded_once(mu, shape):
    """Sequences of one chunk keep 16 bits or more up to the last rounding.  A
    result y + d, |d| <= delta, rounds to within |round(y) - y| + 2 delta of y;
    operands in two pieces are within 2^-16, so terms of five times the result's
    size (of few, random ones) add 2 * 5 * 2^-16 = 1.5e-4, under a tenth of the
    1.7e-3 that rounding itself leaves."""
    x = inputs(*shape, BF16, seed=5)
    want = {"y": ref.scan(x["v"], x["k"], x["q"], x["g"], x["b"], x["S0"])[0]}
    want.update(zip(("dv", "dk", "dq"), ref.scan_grads(x["v"], x["k"], x["q"], x["g"], x["dy"], x["b"], x["S0"], x["dS"])))
    got = {"y": forward(mu, x)[0]}
    got.update(zip(("dv", "dk", "dq"), backward(mu, x)))
    for name, w in want.items():
        once = ref.rel(w.to(BF16), w)
        err = ref.rel(got[name], w)
        print(f"[parity] {name} {err:.2e} rounding {once:.2e}", flush=True)
        assert err <= 1.1 * once, name


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate,state", [(False, False), (True, False), (False, True)])
def test_scan_without_gate_or_states(mu, gate, state, dtype):
    x = inputs(2, 150, 4, 2, 64, 128, dtype, seed=3, gate=gate, state=state)
    check_forward(mu, x)
    check_backward(mu, x)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("resets,decay", [(0.05, 0.1), (0.5, 0.1), (1.0, 0.1), (0.02, 3.0)])
def test_scan_resets(mu, resets, decay, dtype):
    """Packed sequences: -inf starts a new one, at any token, next to each
    other and everywhere."""
    x = inputs(2, 260, 2, 1, 64, 128, dtype, seed=4, resets=resets, decay=decay)
    check_forward(mu, x)
    check_backward(mu, x)


@pytest.mark.parametrize("low", [-torch.finfo(torch.float32).max, -2.0e4, -math.inf])
def test_scan_reset_separates_packed_sequences(mu, low):
    """Two sequences in one row give bit for bit what the reset leaves of
    either: the second's results do not depend on the first's values."""
    x = inputs(1, 100, 2, 1, 64, 128, F32, seed=5, state=False)
    x["g"][:, 37] = low
    y, S = forward(mu, x)
    z = dict(x)
    z["v"] = x["v"].clone()
    z["v"][:, :37] *= -3.0
    y2, S2 = forward(mu, z)
    assert torch.equal(y[:, 37:], y2[:, 37:]) and torch.equal(S, S2)
    assert torch.equal(y[:, :37] * -3.0, y2[:, :37]) or ref.rel(y2[:, :37], -3.0 * y[:, :37].cpu()) < F32_TOL


@pytest.mark.parametrize("decay", [0.0, 1e-4, 2.0, 40.0])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_scan_decay_range(mu, decay, dtype):
    """From no decay at all to states that one token forgets."""
    x = inputs(1, 400, 2, 1, 64, 128, dtype, seed=6, decay=decay)
    check_forward(mu, x)
    check_backward(mu, x)


@pytest.mark.parametrize("shape", [(2, 130, 4, 2, 64, 128), (2, 90, 3, 1, 17, 33), (1, 70, 2, 2, 66, 70)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_scan_sliced_operands(mu, shape, dtype):
    """v, k and q as column ranges of one tensor, three elements off alignment."""
    x = inputs(*shape, dtype, seed=7, sliced=True)
    c = {n: t.cuda() for n, t in x.items()}
    y, S = mu.muon_gated_scan(c["v"], c["k"], c["q"], c["g"], gate=c["b"], S0=c["S0"])
    check_forward(mu, x)
    check_backward(mu, x)
    # the slices themselves (x moved to the GPU tensor by tensor loses them)
    B, T, H, G, P, N = shape
    wide = torch.zeros(B, T, 3 + H * P + 2 * G * N, dtype=dtype, device="cuda")
    v, k, q = wide[..., 3:].split([H * P, G * N, G * N], dim=2)
    v.copy_(c["v"].flatten(2))
    k.copy_(c["k"].flatten(2))
    q.copy_(c["q"].flatten(2))
    v, k, q = v.unflatten(2, (H, P)), k.unflatten(2, (G, N)), q.unflatten(2, (G, N))
    y2, S2 = mu.muon_gated_scan(v, k, q, c["g"], gate=c["b"], S0=c["S0"])
    assert torch.equal(y, y2) and torch.equal(S, S2)
    a = mu.muon_gated_scan_backward(c["v"], c["k"], c["q"], c["g"], c["dy"], gate=c["b"], S0=c["S0"], dS=c["dS"])
    b = mu.muon_gated_scan_backward(v, k, q, c["g"], c["dy"], gate=c["b"], S0=c["S0"], dS=c["dS"])
    assert all(torch.equal(i, j) for i, j in zip(a, b))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off", [1, 2, 3, 5])
def test_scan_at_any_element(mu, off, dtype):
    """Rows of whole 16-byte pieces that start at any element, at an odd stride:
    bit for bit what the same rows give in tensors of their own."""
    B, T, H, G, P, N = 2, 130, 4, 2, 64, 128
    x = {n: t.cuda() for n, t in inputs(B, T, H, G, P, N, dtype, seed=17).items()}
    wide = torch.full((B, T, off + H * P + 2 * G * N + 3), float("nan"), dtype=dtype, device="cuda")
    wide2 = torch.full((B, T, off + H * P), float("nan"), dtype=dtype, device="cuda")
    v, k, q = wide[..., off:off + H * P + 2 * G * N].split([H * P, G * N, G * N], dim=2)
    v, k, q, dy = v.unflatten(2, (H, P)), k.unflatten(2, (G, N)), q.unflatten(2, (G, N)), wide2[..., off:].unflatten(2, (H, P))
    for to, name in ((v, "v"), (k, "k"), (q, "q"), (dy, "dy")):
        to.copy_(x[name])
    rest = dict(gate=x["b"], S0=x["S0"])
    for a, b in zip(mu.muon_gated_scan(v, k, q, x["g"], **rest), mu.muon_gated_scan(x["v"], x["k"], x["q"], x["g"], **rest)):
        assert torch.equal(a, b)
    a = mu.muon_gated_scan_backward(v, k, q, x["g"], dy, dS=x["dS"], **rest)
    b = mu.muon_gated_scan_backward(x["v"], x["k"], x["q"], x["g"], x["dy"], dS=x["dS"], **rest)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_scan_permuted_and_broadcast_operands(mu):
    """Head-major storage, and gates and keys broadcast over tokens (stride 0)."""
    x = inputs(2, 100, 4, 2, 64, 128, BF16, seed=8)
    c = {n: t.cuda() for n, t in x.items()}
    want = mu.muon_gated_scan(c["v"], c["k"], c["q"], c["g"], gate=c["b"], S0=c["S0"])
    hm = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    got = mu.muon_gated_scan(hm(c["v"]), hm(c["k"]), hm(c["q"]), hm(c["g"]), gate=hm(c["b"]), S0=c["S0"])
    assert all(torch.equal(i, j) for i, j in zip(got, want))
    k1, b1 = c["k"][:, :1].expand(-1, 100, -1, -1), c["b"][:, :1].expand(-1, 100, -1)
    want = mu.muon_gated_scan_backward(c["v"], k1.contiguous(), c["q"], c["g"], c["dy"], gate=b1.contiguous())
    got = mu.muon_gated_scan_backward(c["v"], k1, c["q"], c["g"], c["dy"], gate=b1)
    assert all(i is j is None or torch.equal(i, j) for i, j in zip(got, want))


def test_scan_calls_carry_the_state(mu):
    """A sequence in two calls is the sequence in one."""
    x = inputs(1, 333, 3, 1, 64, 128, F32, seed=9)
    y, S = forward(mu, x)
    h = 100
    part = lambda t, s: None if t is None else t[:, s]  # noqa: E731
    a = {n: t if n in ("S0", "dS") else part(t, slice(0, h)).contiguous() for n, t in x.items()}
    y1, S1 = forward(mu, a)
    b = {n: t if n in ("S0", "dS") else part(t, slice(h, None)).contiguous() for n, t in x.items()}
    b["S0"] = S1.cpu()
    y2, S2 = forward(mu, b)
    assert ref.rel(torch.cat([y1, y2], 1), y.cpu()) <= F32_TOL and ref.rel(S2, S.cpu()) <= F32_TOL


def test_scan_gradients_are_differences(mu):
    """float32 gradients against central differences of the float64 forward
    reference: directional derivatives, to the gradients' own tolerance."""
    x = inputs(1, 90, 2, 1, 24, 20, F32, seed=10)
    names = ("v", "k", "q", "g", "b", "S0")
    grads = dict(zip(names, backward(mu, x)))
    gen = torch.Generator().manual_seed(77)

    def loss(z):
        y, S, _ = ref.scan(z["v"], z["k"], z["q"], z["g"], z["b"], z["S0"])
        return float((y * x["dy"].double()).sum() + (S * x["dS"].double()).sum())

    for n in names:
        d = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        diff = (loss({**x, n: x[n].double() + h * d}) - loss({**x, n: x[n].double() - h * d})) / (2 * h)
        g = grads[n].cpu().double()
        assert abs(float((g * d).sum()) - diff) <= F32_TOL * float(g.norm() * d.norm()), n


def test_scan_deterministic_and_workspace_reuse(mu):
    """Bit-identical on repetition, with a workspace full of NaN, given outputs
    and a side stream."""
    x = inputs(1, 1500, 4, 1, 64, 128, BF16, seed=11)
    c = {n: t.cuda() for n, t in x.items()}
    y, S = forward(mu, x)
    g = backward(mu, x)
    nf, nb = mu.muon_gated_scan_workspace_size(x["v"], x["k"]), mu.muon_gated_scan_workspace_size(x["v"], x["k"], backward=True)
    nan = lambda n: torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)  # noqa: E731
    wf, wb = nan(nf), nan(nb)
    Y = torch.full_like(y, float("nan"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, S2 = forward(mu, x, workspace=wf, Y=Y, stream=side)
    side.synchronize()
    assert y2 is Y and torch.equal(y, y2) and torch.equal(S, S2)
    for _ in range(2):
        g2 = backward(mu, x, workspace=wb)
        assert all(torch.equal(i, j) for i, j in zip(g, g2))


def test_scan_empty(mu):
    """No tokens: the state passes through; no sequences: nothing happens."""
    S0 = torch.randn(2, 3, 4, 5, device="cuda")
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    y, S = mu.muon_gated_scan(e(2, 0, 3, 4), e(2, 0, 1, 5), e(2, 0, 1, 5), e(2, 0, 3), S0=S0)
    assert y.numel() == 0 and torch.equal(S, S0)
    y, S = mu.muon_gated_scan(e(2, 0, 3, 4), e(2, 0, 1, 5), e(2, 0, 1, 5), e(2, 0, 3))
    assert torch.equal(S, torch.zeros_like(S0))
    r = mu.muon_gated_scan_backward(e(2, 0, 3, 4), e(2, 0, 1, 5), e(2, 0, 1, 5), e(2, 0, 3), e(2, 0, 3, 4), S0=S0, dS=2 * S0)
    assert torch.equal(r[5], 2 * S0)
    y, S = mu.muon_gated_scan(e(0, 7, 3, 4), e(0, 7, 1, 5), e(0, 7, 1, 5), e(0, 7, 3))
    assert y.numel() == 0 and S.numel() == 0


def test_scan_long_offsets(mu):
    """Operands whose elements lie past 2^31 from the first (a wide row stride,
    one shared buffer): the last token is read and written where it is."""
    T, stride = 40, 60_000_000
    buf = torch.zeros((T - 1) * stride + 64, dtype=BF16, device="cuda")
    gen = torch.Generator().manual_seed(12)
    v = torch.randn(T, 64, generator=gen).to(BF16)
    wide = buf.as_strided((1, T, 1, 64), (0, stride, 0, 1))
    wide.copy_(v.cuda()[None, :, None, :])
    k, q = (torch.randn(1, T, 1, 64, generator=gen).to(BF16) for _ in range(2))
    g = torch.full((1, T, 1), -0.05)
    y, S = mu.muon_gated_scan(wide, k.cuda(), q.cuda(), g.cuda())
    yr, Sr, _ = ref.scan(v[None, :, None, :], k, q, g)
    assert ref.rel(y, yr) <= BF16_TOL and ref.rel(S, Sr) <= F32_TOL


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (3, 4, 2, 64, 128), (2, 6, 3, 40, 72), (2, 2, 1, 17, 5), (1, 2, 1, 130, 99)],
                         ids=str)
@pytest.mark.parametrize("in_place", [True, False])
def test_step(mu, shape, dtype, in_place):
    B, H, G, P, N = shape
    x = inputs(B, 1, H, G, P, N, dtype, seed=13)
    yr, Sr, _ = ref.scan(x["v"], x["k"], x["q"], x["g"], x["b"], x["S0"])
    S = x["S0"].cuda()
    out = None if in_place else torch.full_like(S, float("nan"))
    y, S2 = mu.muon_gated_scan_step(*(x[n][:, 0].cuda() for n in ("v", "k", "q", "g")), S, gate=x["b"][:, 0].cuda(), S_out=out)
    torch.cuda.synchronize()
    assert S2 is (S if in_place else out)
    assert in_place or torch.equal(S.cpu(), x["S0"])
    assert ref.rel(S2, Sr) <= F32_TOL
    assert ref.rel(y, yr[:, 0]) <= (BF16_TOL if dtype == BF16 else F32_TOL)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(13, 24, 1, 60, 128), (12, 24, 2, 64, 99), (300, 4, 1, 17, 72), (64, 2, 2, 130, 36)], ids=str)
def test_step_of_batches(mu, shape, dtype):
    """More than 16,384 rows of states, which take four rows a half-wave."""
    B, H, G, P, N = shape
    x = inputs(B, 1, H, G, P, N, dtype, seed=14)
    yr, Sr, _ = ref.scan(x["v"], x["k"], x["q"], x["g"], x["b"], x["S0"])
    S = x["S0"].cuda()
    y, _ = mu.muon_gated_scan_step(*(x[n][:, 0].cuda() for n in ("v", "k", "q", "g")), S, gate=x["b"][:, 0].cuda())
    assert ref.rel(S, Sr) <= F32_TOL
    assert ref.rel(y, yr[:, 0]) <= (BF16_TOL if dtype == BF16 else F32_TOL)


def test_steps_are_the_scan(mu):
    """Token by token from the state that a prompt's scan left, a reset among
    the tokens, without a gate."""
    x = inputs(2, 90, 4, 2, 64, 128, F32, seed=14, gate=False)
    x["g"][:, 80] = -math.inf
    yr, Sr, _ = ref.scan(x["v"], x["k"], x["q"], x["g"], None, x["S0"])
    head = {n: t if n in ("S0", "dS") or t is None else t[:, :70].contiguous() for n, t in x.items()}
    y, S = forward(mu, head)
    for t in range(70, 90):
        y, S = mu.muon_gated_scan_step(*(x[n][:, t].cuda() for n in ("v", "k", "q", "g")), S)
        assert ref.rel(y, yr[:, t]) <= F32_TOL
    assert ref.rel(S, Sr) <= F32_TOL


def test_scan_in_a_graph(mu):
    """Captured once, replayed on new inputs: forward, backward and step."""
    x = inputs(1, 600, 4, 1, 64, 128, BF16, seed=15)
    c = {n: t.cuda() for n, t in x.items()}
    wf = torch.empty(mu.muon_gated_scan_workspace_size(c["v"], c["k"]), dtype=torch.uint8, device="cuda")
    wb = torch.empty(mu.muon_gated_scan_workspace_size(c["v"], c["k"], backward=True), dtype=torch.uint8, device="cuda")

    def call():
        r = mu.muon_gated_scan(c["v"], c["k"], c["q"], c["g"], gate=c["b"], S0=c["S0"], workspace=wf)
        return r + mu.muon_gated_scan_backward(c["v"], c["k"], c["q"], c["g"], c["dy"], gate=c["b"], S0=c["S0"], dS=c["dS"],
                                               workspace=wb)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in (16, 17, 18):
        z = inputs(1, 600, 4, 1, 64, 128, BF16, seed=seed)
        for n in c:
            c[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def _random_case(seed):
    gen = torch.Generator().manual_seed(seed)
    ri = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=gen))  # noqa: E731
    G = ri(1, 3)
    return (ri(1, 3), ri(1, 400), G * ri(1, 4), G, ri(1, 140), ri(1, 128)), bool(ri(0, 1)), bool(ri(0, 1)), ri(0, 2) * 0.02, \
        bool(ri(0, 1)), [0.01, 0.2, 2.0][ri(0, 2)]


@pytest.mark.parametrize("seed", range(10))
def test_scan_random_cases(mu, seed):
    shape, gate, state, resets, sliced, decay = _random_case(seed)
    print(f"[case] {shape} gate {gate} state {state} resets {resets} decay {decay}", flush=True)
    x = inputs(*shape, BF16 if seed % 2 else F32, seed=seed, gate=gate, state=state, resets=resets, decay=decay, sliced=sliced)
    check_forward(mu, x)
    check_backward(mu, x)
