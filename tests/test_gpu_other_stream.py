"""Calls on another stream than torch's current one: whatever a call makes for
itself comes from that stream's memory.  A block of the current stream's memory
may have been freed while kernels queued there still use it, and nothing
orders them before a kernel of the other stream.  Shown by where the memory is
asked for; nothing here races."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spectral_optimizer_ssm_amd as mu
    mu.lib()
    return mu


def scan_inputs(tokens):
    gen = torch.Generator().manual_seed(41)
    rn = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    B, H, G, P, N = 2, 4, 2, 64, 128
    lead = (B, tokens) if tokens else (B,)
    return dict(v=rn(*lead, H, P), k=rn(*lead, G, N), q=rn(*lead, G, N), g=-rn(*lead, H).abs(), b=rn(*lead, H), S=rn(B, H, P, N),
                dy=rn(*lead, H, P))


def calls(mu):
    """name: (call(stream), its tensors) of every entry point that makes tensors."""
    x, one = scan_inputs(150), scan_inputs(0)
    X, w = torch.randn(40, 96, device="cuda"), torch.rand(96, device="cuda")
    _, mean, rstd = mu.muon_layer_norm(X, w)
    mats = torch.randn(2, 64, 128, device="cuda").bfloat16()
    facs = [torch.randn(3, m, 8, device="cuda").bfloat16() for m in (64, 128)]
    seqs = [torch.randn(2, 5, m, 8, device="cuda").bfloat16() for m in (64, 128)]

    def step(s):
        group = mu.MuonGroup(W=torch.zeros(2, 64, 128, device="cuda"), M=torch.zeros(2, 64, 128, device="cuda"), G=mats, lr=0.1, beta=0.9)
        torch.cuda.synchronize()
        return lambda: [mu.muon_step([group], stream=s)]

    def momentum(s):
        M = torch.zeros(2, 64, 128, device="cuda")
        torch.cuda.synchronize()
        return lambda: [M, mu.muon_ssm_momentum(*seqs, M, stream=s)][:1]

    def orthogonalize(s):
        O = torch.empty_like(mats)
        return lambda: [O, mu.muon_ns_orthogonalize(mats, O, stream=s)][:1]

    def one_step(s):
        S = one["S"].clone()
        torch.cuda.synchronize()
        return lambda: list(mu.muon_gated_scan_step(one["v"], one["k"], one["q"], one["g"], S, gate=one["b"], stream=s))

    return {
        "scan": lambda s: lambda: list(mu.muon_gated_scan(x["v"], x["k"], x["q"], x["g"], gate=x["b"], S0=x["S"], stream=s)),
        "scan_backward": lambda s: lambda: list(mu.muon_gated_scan_backward(x["v"], x["k"], x["q"], x["g"], x["dy"], gate=x["b"],
                                                                            S0=x["S"], stream=s)),
        "scan_step": one_step,
        "norm": lambda s: lambda: list(mu.muon_layer_norm(X, w, stream=s)),
        "norm_backward": lambda s: lambda: list(mu.muon_layer_norm_backward(X, X, w, mean, rstd, stream=s)),
        "muon_step": step,
        "ns_orthogonalize": orthogonalize,
        "ns_factored": lambda s: lambda: [mu.muon_ns_factored(*facs, stream=s)],
        "ssm_momentum": momentum,
        "spectral_diag": lambda s: lambda: list(mu.muon_spectral_diag(mats, iters=8, stream=s).values()),
    }


@pytest.mark.parametrize("name", ["scan", "scan_backward", "scan_step", "norm", "norm_backward", "muon_step", "ns_orthogonalize",
                                  "ns_factored", "ssm_momentum", "spectral_diag"])
def test_new_tensors_come_from_the_streams_memory(mu, monkeypatch, name):
    make = calls(mu)[name]
    want = make(None)()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call = make(side)
    torch.cuda.synchronize()
    asked, recorded = [], []
    empty, empty_like, record = torch.empty, torch.empty_like, torch.Tensor.record_stream

    def spy(f):
        def made(*a, **kw):
            asked.append(torch.cuda.current_stream())
            return f(*a, **kw)
        return made

    def record_stream(t, s):
        recorded.append((t.data_ptr(), s))
        return record(t, s)

    with monkeypatch.context() as m:
        m.setattr(torch, "empty", spy(empty))
        m.setattr(torch, "empty_like", spy(empty_like))
        m.setattr(torch.Tensor, "record_stream", record_stream)
        got = call()
    here = torch.cuda.current_stream()
    side.synchronize()
    assert here != side and asked and all(s == side for s in asked), asked
    # what is handed back is not given out again before the caller's stream is done with it
    for t in got:
        if t is not None and name not in ("ns_orthogonalize", "ssm_momentum"):
            assert (t.data_ptr(), here) in recorded
    if name != "muon_step":   # (there what is handed back is the workspace)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))


def test_given_tensors_are_recorded(mu, monkeypatch):
    """Outputs, states and workspaces of the caller's are in use by the other stream."""
    x, one = scan_inputs(150), scan_inputs(0)
    Y, ws = torch.empty_like(x["v"]), torch.empty(mu.muon_gated_scan_workspace_size(x["v"], x["k"]), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side, recorded, record = torch.cuda.Stream(), [], torch.Tensor.record_stream

    def record_stream(t, s):
        recorded.append((t.data_ptr(), s))
        return record(t, s)

    with monkeypatch.context() as m:
        m.setattr(torch.Tensor, "record_stream", record_stream)
        mu.muon_gated_scan(x["v"], x["k"], x["q"], x["g"], Y=Y, workspace=ws, stream=side)
        mu.muon_gated_scan_step(one["v"], one["k"], one["q"], one["g"], one["S"], stream=side)
    side.synchronize()
    for t in (Y, ws, one["S"]):
        assert (t.data_ptr(), side) in recorded
