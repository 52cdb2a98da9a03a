"""The embedding, the group norm and the token log probabilities in HIP graphs (every
replay against the eager call), on other streams, and two calls at once."""
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


def inputs(seed, tokens=700, vocab=900, n=192, dtype=BF16):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    ids = torch.randint(-2, vocab, (tokens,), generator=gen)
    ids[torch.rand(tokens, generator=gen) < 0.4] = 7    # one id often
    return dict(ids=ids.cuda(), table=rn(vocab, n).cuda(), dy=rn(tokens, n).to(dtype).cuda(), z=rn(tokens, n).to(dtype).cuda(),
                w=rn(n).cuda(), x=(2 * rn(tokens, vocab)).to(dtype).cuda(), dl=rn(tokens).cuda())


def passes(mu, i, **kw):
    """name: one pass, a list of tensors."""
    def norm():
        y, _, rstd = mu.muon_group_norm(i["dy"], 3, i["w"], gate=i["z"], **kw)
        return [y, rstd]

    def norm_backward():
        rstd = torch.ones(i["dy"].shape[0], 3, device="cuda")
        return list(mu.muon_group_norm_backward(i["dy"], i["z"], 3, i["w"], None, None, rstd, gate=i["dy"], **kw))[:3]

    def logprobs():
        return list(mu.muon_token_logprobs(i["x"], i["ids"], top=9, **kw))

    def few_logprobs():
        return list(mu.muon_token_logprobs(i["x"].reshape(5, -1), top=30, **kw))[1:]

    def logprobs_backward():
        stats = torch.stack([i["x"].float().max(1).values, torch.full((i["x"].shape[0],), 3.0, device="cuda")], 1)
        return [mu.muon_token_logprobs_backward(i["x"], i["ids"], stats, i["dl"], entropy=i["dl"], dentropy=i["dl"], **kw)]

    return {"embedding": lambda: [mu.muon_embedding(i["table"], i["ids"], dtype=BF16, **kw)],
            "embedding_backward": lambda: [mu.muon_embedding_backward(i["dy"], i["ids"], i["table"].shape[0], **kw)],
            "group_norm": norm, "group_norm_backward": norm_backward, "logprobs": logprobs, "few_logprobs": few_logprobs,
            "logprobs_backward": logprobs_backward}


NAMES = ["embedding", "embedding_backward", "group_norm", "group_norm_backward", "logprobs", "few_logprobs", "logprobs_backward"]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", NAMES)
def test_graph(mu, name, dtype):
    """Captured once, replayed on new inputs with eager work between."""
    i = inputs(1, dtype=dtype)
    call = passes(mu, i)[name]
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in range(2, 6):
        for k, v in inputs(seed, dtype=dtype).items():
            i[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_graph_of_a_training_step(mu):
    """Forward and backward in one graph, the table's gradient accumulated over two
    replays' worth of steps."""
    i = inputs(1)
    total = torch.zeros(900, 192, device="cuda")

    def step(acc):
        x = mu.muon_embedding(i["table"], i["ids"], dtype=BF16)
        y, _, rstd = mu.muon_group_norm(x, 3, i["w"], gate=i["z"])
        logp, H, stats, _, _ = mu.muon_token_logprobs(i["x"], i["ids"])
        dl = mu.muon_token_logprobs_backward(i["x"], i["ids"], stats, i["dl"], entropy=H, dentropy=i["dl"])
        dx, _, dw, _ = mu.muon_group_norm_backward(i["dy"], x, 3, i["w"], None, None, rstd, gate=i["z"])
        mu.muon_embedding_backward(dx, i["ids"], 900, dtable=acc, accumulate=True)
        return y, logp, dl, dw

    step(total.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(total)
    total.zero_()
    want = torch.zeros_like(total)
    for seed in range(2, 6):
        for k, v in inputs(seed).items():
            i[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        eager = step(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)) and torch.equal(total, want), seed


@pytest.mark.parametrize("name", NAMES)
def test_other_stream(mu, monkeypatch, name):
    """What a call on another stream makes for itself comes from that stream's memory, and
    what it gives is recorded on the caller's."""
    i = inputs(3)
    want = passes(mu, i)[name]()
    side = torch.cuda.Stream()
    call = passes(mu, i, stream=side)[name]
    torch.cuda.synchronize()
    recorded, record = [], torch.Tensor.record_stream
    asked, empty, empty_like = [], torch.empty, torch.empty_like

    def spy(f):
        def made(*a, **kw):
            asked.append(torch.cuda.current_stream())
            return f(*a, **kw)
        return made

    def record_stream(t, s):
        recorded.append((t.data_ptr(), s))
        return record(t, s)

    with monkeypatch.context() as m:
        m.setattr(torch.Tensor, "record_stream", record_stream)
        if name not in ("group_norm_backward", "logprobs_backward"):   # (there the test itself makes tensors)
            m.setattr(torch, "empty", spy(empty))
            m.setattr(torch, "empty_like", spy(empty_like))
            torch.cuda.synchronize()
        else:
            torch.cuda.synchronize()
        got = call()
    here = torch.cuda.current_stream()
    torch.cuda.synchronize()
    assert all(s == side for s in asked)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and (a.data_ptr(), here) in recorded


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(mu, name):
    """Two calls with workspaces of their own, interleaved on two streams."""
    a, b = inputs(4), inputs(5)
    want = [passes(mu, i)[name]() for i in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got = []
        for i, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(passes(mu, i)[name]())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))


def test_given_workspaces(mu):
    """A workspace of the caller's, full of anything, one for every call in turn."""
    i = inputs(6)
    ws = torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")
    want = passes(mu, i)
    for _ in range(2):
        assert torch.equal(mu.muon_embedding_backward(i["dy"], i["ids"], 900, workspace=ws), want["embedding_backward"]()[0])
        for a, b in zip(mu.muon_token_logprobs(i["x"].reshape(5, -1), top=30, workspace=ws)[1:], want["few_logprobs"]()):
            assert torch.equal(a, b)
        rstd = torch.ones(700, 3, device="cuda")
        got = mu.muon_group_norm_backward(i["dy"], i["z"], 3, i["w"], None, None, rstd, gate=i["dy"], workspace=ws)
        for a, b in zip(got[:3], want["group_norm_backward"]()):
            assert torch.equal(a, b)


def test_two_graphs_share_a_workspace(mu):
    """Captured with one workspace between them and replayed in turn."""
    ws = torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")
    sets = [inputs(7), inputs(8)]

    def step(i, **kw):
        few = mu.muon_token_logprobs(i["x"].reshape(5, -1), top=30, **kw)[1:]
        dx = mu.muon_group_norm_backward(i["dy"], i["z"], 3, i["w"], None, None, torch.ones(700, 3, device="cuda"), gate=i["dy"], **kw)[:3]
        return [*few, *dx, mu.muon_embedding_backward(dx[0], i["ids"], 900, **kw)]

    graphs, outs = [], []
    for i in sets:
        step(i, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(i, workspace=ws))
    for seed in range(9, 12):
        for k, i in enumerate(sets):
            for name, v in inputs(seed + 10 * k).items():
                i[name].copy_(v)
        for g in (*graphs, *graphs[::-1]):
            g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in out] for out in outs]
        for i, out in zip(sets, got):
            assert all(torch.equal(a, b) for a, b in zip(out, step(i))), seed
