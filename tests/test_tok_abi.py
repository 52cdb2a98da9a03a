"""Refusals of the embedding, the group norm and the token log probabilities, at
the C ABI and in the binding: nothing is enqueued on a bad argument (no GPU
needed: pointers are made up and never read)."""
import os
import struct

import pytest

torch = pytest.importorskip("torch")

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
BIG = 1 << 40
A = 1 << 36            # made-up device addresses, far apart
ADDR = {n: A * (i + 1) for i, n in enumerate(("table", "ids", "Y", "dY", "dtable", "ws", "X", "Z", "w", "b", "mean", "rstd", "dX", "dZ",
                                              "dw", "db", "logp", "H", "stats", "top", "lp", "dlp", "dH"))}


@pytest.fixture(scope="module")
def mu():
    import spectral_optimizer_ssm_amd as mu
    if not os.path.exists(mu.binding.LIB_PATH):
        pytest.fail("libmuon.so is not built: run python -m spectral_optimizer_ssm_amd.build")
    mu.lib()
    return mu


def ids(p=ADDR["ids"], bits=64, run=1 << 20, stride=0, step=1):
    return struct.pack("@Pi4xqqq", p or 0, bits, run, stride, step)


BAD_IDS = [dict(ids=None), dict(ids=ids(p=0)), dict(ids=ids(bits=16)), dict(ids=ids(p=ADDR["ids"] + 4)), dict(ids=ids(bits=32, p=ADDR["ids"] + 2)),
           dict(ids=ids(run=0)), dict(ids=ids(stride=-1)), dict(ids=ids(step=-1)), dict(ids=ids(run=2, stride=1 << 60)),
           dict(ids=ids(step=1 << 60))]


def embed(mu, **kw):
    a = dict(table=ADDR["table"], tt=0, ldt=768, vocab=100, n=768, ids=ids(), tokens=50, scale=1.0, Y=ADDR["Y"], dt=1, ldy=768, **{})
    a.update(kw)
    return mu.lib().muon_embedding(a["table"], a["tt"], a["ldt"], a["vocab"], a["n"], a["ids"], a["tokens"], a["scale"], a["Y"], a["dt"],
                                   a["ldy"], None)


@pytest.mark.parametrize("bad,expect", [
    (dict(tt=2), EINVAL), (dict(dt=-1), EINVAL), (dict(vocab=0), EINVAL), (dict(n=0), EINVAL), (dict(tokens=-1), EINVAL),
    (dict(tokens=(1 << 30) + 1), EUNSUPPORTED), (dict(vocab=(1 << 30) + 1), EUNSUPPORTED),
    (dict(n=(1 << 21) + 1, ldt=1 << 22, ldy=1 << 22), EUNSUPPORTED), (dict(tokens=1 << 30, n=2048, ldt=2048, ldy=2048), EUNSUPPORTED),
    (dict(vocab=1 << 30, n=2048, ldt=2048, ldy=2048), EUNSUPPORTED),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(ldt=767), EINVAL), (dict(ldy=767), EINVAL),
    (dict(ldy=1 << 58), EINVAL), (dict(table=None), EINVAL), (dict(Y=None), EINVAL), (dict(table=ADDR["table"] + 2), EINVAL),
    (dict(Y=ADDR["Y"] + 1), EINVAL), (dict(Y=ADDR["table"]), EINVAL), (dict(Y=ADDR["table"] + 4 * 768 * 99), EINVAL),
    (dict(Y=ADDR["ids"] + 8), EINVAL), *[(b, EINVAL) for b in BAD_IDS],
], ids=lambda v: None if isinstance(v, int) else str(v)[:60])
def test_embedding_refusals(mu, bad, expect):
    assert embed(mu, **bad) == expect


def embed_bwd(mu, **kw):
    a = dict(dY=ADDR["dY"], dt=1, lddy=768, ids=ids(), tokens=50, scale=1.0, vocab=100, n=768, dtable=ADDR["dtable"], tt=0, acc=0,
             ws=ADDR["ws"], nbytes=BIG)
    a.update(kw)
    return mu.lib().muon_embedding_backward(a["dY"], a["dt"], a["lddy"], a["ids"], a["tokens"], a["scale"], a["vocab"], a["n"], a["dtable"],
                                            a["tt"], a["acc"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("bad,expect", [
    (dict(tt=2), EINVAL), (dict(dt=7), EINVAL), (dict(vocab=0), EINVAL), (dict(n=0), EINVAL), (dict(tokens=-1), EINVAL),
    (dict(tokens=(1 << 30) + 1), EUNSUPPORTED), (dict(n=(1 << 21) + 1, lddy=1 << 22), EUNSUPPORTED),
    (dict(acc=2), EINVAL), (dict(acc=1, tt=1), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(lddy=700), EINVAL),
    (dict(dY=None), EINVAL), (dict(dY=ADDR["dY"] + 1), EINVAL), (dict(dtable=None), EINVAL), (dict(dtable=ADDR["dtable"] + 2), EINVAL),
    (dict(ws=None), EWORKSPACE), (dict(ws=ADDR["ws"] + 8), EWORKSPACE), (dict(nbytes=1000), EWORKSPACE),
    (dict(dtable=ADDR["dY"]), EINVAL), (dict(ws=ADDR["dY"] + 16), EINVAL), (dict(ws=ADDR["dtable"]), EINVAL),
    (dict(dtable=ADDR["ids"]), EINVAL), (dict(tokens=0, ws=ADDR["dtable"]), EINVAL), *[(b, EINVAL) for b in BAD_IDS],
], ids=lambda v: None if isinstance(v, int) else str(v)[:60])
def test_embedding_backward_refusals(mu, bad, expect):
    assert embed_bwd(mu, **bad) == expect


def norm(mu, **kw):
    a = dict(X=ADDR["X"], ldx=768, Z=ADDR["Z"], ldz=768, dt=1, rows=10, groups=3, w_=256, w=ADDR["w"], b=ADDR["b"], eps=1e-5, center=1,
             gate=0, Y=ADDR["Y"], ldy=768, mean=ADDR["mean"], rstd=ADDR["rstd"])
    a.update(kw)
    return mu.lib().muon_group_norm(a["X"], a["ldx"], a["Z"], a["ldz"], a["dt"], a["rows"], a["groups"], a["w_"], a["w"], a["b"], a["eps"],
                                    a["center"], a["gate"], a["Y"], a["ldy"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("bad,expect", [
    (dict(dt=3), EINVAL), (dict(rows=-1), EINVAL), (dict(groups=0), EINVAL), (dict(w_=0), EINVAL), (dict(rows=1 << 31), EUNSUPPORTED),
    (dict(rows=1 << 30, groups=4), EUNSUPPORTED), (dict(groups=65536), EUNSUPPORTED), (dict(groups=4096, w_=1 << 20), EUNSUPPORTED),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(center=2), EINVAL), (dict(gate=-1), EINVAL), (dict(gate=4), EINVAL),
    (dict(gate=2), EINVAL), (dict(gate=3), EINVAL), (dict(Z=None), EINVAL), (dict(gate=1, Z=None), EINVAL), (dict(ldx=767), EINVAL),
    (dict(ldz=767), EINVAL), (dict(ldy=700), EINVAL), (dict(X=None), EINVAL), (dict(Y=None), EINVAL), (dict(X=ADDR["X"] + 1), EINVAL),
    (dict(Z=ADDR["Z"] + 1), EINVAL), (dict(Y=ADDR["Y"] + 1), EINVAL), (dict(w=ADDR["w"] + 2), EINVAL), (dict(b=ADDR["b"] + 1), EINVAL),
    (dict(mean=ADDR["mean"] + 2), EINVAL), (dict(rstd=ADDR["rstd"] + 2), EINVAL), (dict(Y=ADDR["X"]), EINVAL), (dict(Y=ADDR["Z"]), EINVAL),
    (dict(mean=ADDR["rstd"]), EINVAL), (dict(rstd=ADDR["w"]), EINVAL), (dict(ldx=1 << 60), EINVAL),
], ids=lambda v: None if isinstance(v, int) else str(v)[:60])
def test_group_norm_refusals(mu, bad, expect):
    assert norm(mu, **bad) == expect


def norm_bwd(mu, **kw):
    a = dict(dY=ADDR["dY"], lddy=768, X=ADDR["X"], ldx=768, Z=ADDR["Z"], ldz=768, dt=1, rows=10, groups=3, w_=256, w=ADDR["w"], b=ADDR["b"],
             mean=ADDR["mean"], rstd=ADDR["rstd"], gate=0, dX=ADDR["dX"], lddx=768, dZ=ADDR["dZ"], lddz=768, dw=ADDR["dw"], db=ADDR["db"],
             ws=ADDR["ws"], nbytes=BIG)
    a.update(kw)
    return mu.lib().muon_group_norm_backward(
        a["dY"], a["lddy"], a["X"], a["ldx"], a["Z"], a["ldz"], a["dt"], a["rows"], a["groups"], a["w_"], a["w"], a["b"], a["mean"], a["rstd"],
        a["gate"], a["dX"], a["lddx"], a["dZ"], a["lddz"], a["dw"], a["db"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("bad,expect", [
    (dict(dt=3), EINVAL), (dict(rows=-1), EINVAL), (dict(groups=0), EINVAL), (dict(rows=1 << 30, groups=4), EUNSUPPORTED),
    (dict(gate=5), EINVAL), (dict(gate=2), EINVAL), (dict(gate=2, Z=None), EINVAL), (dict(Z=None), EINVAL), (dict(dZ=None), EINVAL),
    (dict(lddy=1), EINVAL), (dict(ldx=1), EINVAL), (dict(ldz=1), EINVAL), (dict(lddx=1), EINVAL), (dict(lddz=1), EINVAL),
    (dict(dY=None), EINVAL), (dict(X=None), EINVAL), (dict(dX=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dX=ADDR["dX"] + 1), EINVAL),
    (dict(dZ=ADDR["dZ"] + 1), EINVAL), (dict(dw=ADDR["dw"] + 2), EINVAL), (dict(mean=ADDR["mean"] + 1), EINVAL),
    (dict(ws=None), EWORKSPACE), (dict(nbytes=16), EWORKSPACE), (dict(ws=ADDR["ws"] + 8), EWORKSPACE), (dict(dX=ADDR["X"]), EINVAL),
    (dict(dX=ADDR["dY"] + 64), EINVAL), (dict(dZ=ADDR["dX"]), EINVAL), (dict(dZ=ADDR["Z"]), EINVAL), (dict(dw=ADDR["db"]), EINVAL),
    (dict(dw=ADDR["w"]), EINVAL),
], ids=lambda v: None if isinstance(v, int) else str(v)[:60])
def test_group_norm_backward_refusals(mu, bad, expect):
    assert norm_bwd(mu, **bad) == expect


def logp(mu, **kw):
    a = dict(X=ADDR["X"], ldx=1000, dt=1, rows=10, vocab=1000, scale=1.0, ids=ids(), logp=ADDR["logp"], H=ADDR["H"], stats=ADDR["stats"], k=5,
             top=ADDR["top"], lp=ADDR["lp"], ws=ADDR["ws"], nbytes=BIG)
    a.update(kw)
    return mu.lib().muon_token_logprobs(a["X"], a["ldx"], a["dt"], a["rows"], a["vocab"], a["scale"], a["ids"], a["logp"], a["H"], a["stats"],
                                        a["k"], a["top"], a["lp"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("bad,expect", [
    (dict(dt=4), EINVAL), (dict(rows=-1), EINVAL), (dict(vocab=0), EINVAL), (dict(k=-1), EINVAL), (dict(k=65), EUNSUPPORTED),
    (dict(rows=1 << 31), EUNSUPPORTED), (dict(vocab=(1 << 27) + 1), EUNSUPPORTED),
    (dict(rows=1 << 20, vocab=(1 << 20) + 1), EUNSUPPORTED), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(ldx=999), EINVAL), (dict(X=None), EINVAL),
    (dict(X=ADDR["X"] + 1), EINVAL), (dict(logp=ADDR["logp"] + 1), EINVAL), (dict(H=ADDR["H"] + 2), EINVAL),
    (dict(stats=ADDR["stats"] + 1), EINVAL), (dict(top=None), EINVAL), (dict(lp=None), EINVAL), (dict(k=0), EINVAL),
    (dict(top=ADDR["top"] + 1), EINVAL), (dict(ws=None), EWORKSPACE), (dict(ws=ADDR["ws"] + 4), EWORKSPACE), (dict(nbytes=8), EWORKSPACE),
    (dict(logp=ADDR["X"]), EINVAL), (dict(H=ADDR["logp"]), EINVAL), (dict(stats=ADDR["ids"]), EINVAL), (dict(ws=ADDR["X"] + 16), EINVAL),
    (dict(lp=ADDR["top"]), EINVAL), *[(b, EINVAL) for b in BAD_IDS],
], ids=lambda v: None if isinstance(v, int) else str(v)[:60])
def test_logprobs_refusals(mu, bad, expect):
    assert logp(mu, **bad) == expect


def logp_bwd(mu, **kw):
    a = dict(X=ADDR["X"], ldx=1000, dt=1, rows=10, vocab=1000, scale=1.0, ids=ids(), stats=ADDR["stats"], dlp=ADDR["dlp"], sdlp=1, H=ADDR["H"],
             dH=ADDR["dH"], sdh=1, dX=ADDR["dX"], lddx=1000)
    a.update(kw)
    return mu.lib().muon_token_logprobs_backward(a["X"], a["ldx"], a["dt"], a["rows"], a["vocab"], a["scale"], a["ids"], a["stats"], a["dlp"],
                                                 a["sdlp"], a["H"], a["dH"], a["sdh"], a["dX"], a["lddx"], None)


@pytest.mark.parametrize("bad,expect", [
    (dict(dt=4), EINVAL), (dict(rows=-1), EINVAL), (dict(vocab=0), EINVAL), (dict(rows=1 << 20, vocab=(1 << 20) + 1), EUNSUPPORTED),
    (dict(scale=0.0), EINVAL), (dict(ldx=999), EINVAL), (dict(lddx=999), EINVAL), (dict(X=None), EINVAL), (dict(dX=None), EINVAL),
    (dict(stats=None), EINVAL), (dict(stats=ADDR["stats"] + 2), EINVAL), (dict(dlp=ADDR["dlp"] + 2), EINVAL), (dict(sdlp=-1), EINVAL),
    (dict(sdh=-1), EINVAL), (dict(sdlp=1 << 60), EINVAL), (dict(H=None), EINVAL), (dict(dX=ADDR["dX"] + 1), EINVAL),
    (dict(dX=ADDR["X"] + 2), EINVAL), (dict(dX=ADDR["X"], lddx=1001), EINVAL), (dict(dX=ADDR["stats"]), EINVAL),
    (dict(dX=ADDR["dlp"]), EINVAL), (dict(dX=ADDR["H"]), EINVAL), (dict(dX=ADDR["dH"]), EINVAL), *[(b, EINVAL) for b in BAD_IDS],
], ids=lambda v: None if isinstance(v, int) else str(v)[:60])
def test_logprobs_backward_refusals(mu, bad, expect):
    assert logp_bwd(mu, **bad) == expect


def test_nothing_to_do(mu):
    L = mu.lib()
    assert embed(mu, tokens=0, table=None, Y=None, ids=None) == 0
    assert embed_bwd(mu, tokens=0, acc=1, dY=None, ids=None) == 0
    assert norm(mu, rows=0, X=None, Y=None) == 0
    assert norm_bwd(mu, rows=0, dY=None, X=None, Z=None, dX=None, dZ=None, rstd=None, dw=None, db=None, ws=None, nbytes=0) == 0
    assert logp(mu, rows=0, X=None, ws=None) == 0 and logp_bwd(mu, rows=0, X=None, dX=None) == 0
    assert L.muon_embedding_backward_workspace_size(10, 0, 8) == 0 and L.muon_embedding_backward_workspace_size(10, 100, 8) > 0
    assert L.muon_group_norm_backward_workspace_size(10, 0, 8, 1) == 0 and L.muon_group_norm_backward_workspace_size(10, 2, 8, 5) == 0
    assert L.muon_group_norm_backward_workspace_size(10, 2, 64, 1) >= 2 * 128 * 4
    assert L.muon_token_logprobs_workspace_size(10, 0, 1, 0) == 0 and L.muon_token_logprobs_workspace_size(10, 1000, 1, 65) == 0
    assert L.muon_token_logprobs_workspace_size(10, 1000, 1, 0) > 0


def test_ids_match_the_header(tmp_path, mu):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "muon.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu %zu", sizeof(muon_ids), offsetof(muon_ids, bits), offsetof(muon_ids, run),'
                   ' offsetof(muon_ids, stride), offsetof(muon_ids, step));return 0;}\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "t")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "t")], capture_output=True, text=True).stdout.split()]
    assert got == [mu.binding._IDS.size, 8, 16, 24, 32]


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
@pytest.fixture
def on_cpu(mu, monkeypatch):
    """Everything is taken to be on the GPU; a call that gets past the checks fails for want of it."""
    B = mu.binding
    if B.torch is None:
        B._load_torch()
    monkeypatch.setattr(B, "_device_index", lambda: 0)
    monkeypatch.setattr(B, "_where", lambda t, name, index: None)
    return mu


Z = torch.zeros
I = lambda *s: torch.zeros(*s, dtype=torch.int64)  # noqa: E731,E741


@pytest.mark.parametrize("call,error", [
    (lambda m: m.muon_embedding(Z(4, 8, 2), I(3)), ValueError), (lambda m: m.muon_embedding(Z(4, 8).half(), I(3)), TypeError),
    (lambda m: m.muon_embedding(Z(4, 8), Z(3)), TypeError), (lambda m: m.muon_embedding(Z(4, 8), I(3).short()), TypeError),
    (lambda m: m.muon_embedding(Z(8, 4).T, I(3)), ValueError), (lambda m: m.muon_embedding(Z(4, 8), I(3), Y=Z(3, 9)), ValueError),
    (lambda m: m.muon_embedding(Z(4, 8), I(3), dtype=torch.bfloat16, Y=Z(3, 8)), TypeError),
    (lambda m: m.muon_embedding(Z(4, 8), I(2, 3, 4, 5)[:, ::2, ::2, ::2]), ValueError),
    (lambda m: m.muon_embedding_backward(Z(3, 8), I(4), 10), ValueError), (lambda m: m.muon_embedding_backward(Z(3, 8).half(), I(3), 10), TypeError),
    (lambda m: m.muon_embedding_backward(Z(3, 8), I(3), 10, accumulate=True), ValueError),
    (lambda m: m.muon_embedding_backward(Z(3, 8), I(3), 10, dtable=Z(9, 8)), ValueError),
    (lambda m: m.muon_embedding_backward(Z(3, 8), I(3), 10, dtable=Z(8, 10).T), ValueError),
    (lambda m: m.muon_embedding_backward(Z(3, 8), I(3), 10, dtype=torch.bfloat16, dtable=Z(10, 8)), TypeError),
    (lambda m: m.muon_embedding_backward(Z(3, 8), I(3), 0), RuntimeError),
    (lambda m: m.muon_embedding_backward(Z(3, 8), I(3), 10, dtable=Z(10, 8), workspace=Z(9)), TypeError),
    (lambda m: m.muon_group_norm(Z(3, 8), 3), ValueError), (lambda m: m.muon_group_norm(Z(3, 8), 0), ValueError),
    (lambda m: m.muon_group_norm(Z(3, 8).half(), 2), TypeError), (lambda m: m.muon_group_norm(Z(3, 8), 2, gate=Z(3, 9)), ValueError),
    (lambda m: m.muon_group_norm(Z(3, 8), 2, gate=Z(3, 8).bfloat16()), TypeError),
    (lambda m: m.muon_group_norm(Z(3, 8), 2, activation="relu"), ValueError),
    (lambda m: m.muon_group_norm(Z(3, 8), 2, gate=Z(3, 8), activation="none"), ValueError),
    (lambda m: m.muon_group_norm(Z(3, 8), 2, weight=Z(4)), ValueError), (lambda m: m.muon_group_norm(Z(3, 8), 2, bias=Z(8).bfloat16()), TypeError),
    (lambda m: m.muon_group_norm(Z(8, 3).T, 2), ValueError), (lambda m: m.muon_group_norm(Z(3, 8), 2, Y=Z(3, 7)), ValueError),
    (lambda m: m.muon_group_norm_backward(Z(3, 7), Z(3, 8), 2, None, None, None, Z(3, 2)), ValueError),
    (lambda m: m.muon_group_norm_backward(Z(3, 8), Z(3, 8), 2, None, None, None, Z(3)), ValueError),
    (lambda m: m.muon_group_norm_backward(Z(3, 8), Z(3, 8), 2, None, None, None, Z(3, 2), center=True), ValueError),
    (lambda m: m.muon_group_norm_backward(Z(3, 8).bfloat16(), Z(3, 8), 2, None, None, None, Z(3, 2)), TypeError),
    (lambda m: m.muon_token_logprobs(Z(3, 8).half(), I(3)), TypeError), (lambda m: m.muon_token_logprobs(Z(3, 8), I(4)), ValueError),
    (lambda m: m.muon_token_logprobs(Z(3, 8), Z(3)), TypeError), (lambda m: m.muon_token_logprobs(Z(8, 3).T, I(8)), ValueError),
    (lambda m: m.muon_token_logprobs(Z(3, 8), I(3), top=65), RuntimeError),
    (lambda m: m.muon_token_logprobs_backward(Z(3, 8), I(3), Z(3), Z(3)), ValueError),
    (lambda m: m.muon_token_logprobs_backward(Z(3, 8), I(3), Z(3, 2), Z(4)), ValueError),
    (lambda m: m.muon_token_logprobs_backward(Z(3, 8), I(3), Z(3, 2), Z(3).double()), TypeError),
    (lambda m: m.muon_token_logprobs_backward(Z(3, 8), None, Z(3, 2), Z(3)), ValueError),
    (lambda m: m.muon_token_logprobs_backward(Z(3, 8), I(3), Z(3, 2), Z(3), dentropy=Z(3)), ValueError),
    (lambda m: m.muon_token_logprobs_backward(Z(2, 3, 8), I(2, 3), Z(2, 3, 2), Z(3, 2).T), ValueError),
    (lambda m: m.muon_token_logprobs_backward(Z(3, 8), I(3), Z(3, 2), Z(3), dlogits=Z(3, 8).bfloat16()), TypeError),
])
def test_binding_refuses(on_cpu, call, error, monkeypatch):
    # outputs that the binding makes for itself would need the GPU: refusals come first
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(error):
        call(on_cpu)


def test_binding_refuses_the_cpu(mu, monkeypatch):
    B = mu.binding
    if B.torch is None:
        B._load_torch()
    monkeypatch.setattr(B, "_device_index", lambda: 0)
    for call in (lambda: mu.muon_embedding(Z(4, 8), I(3)), lambda: mu.muon_embedding_backward(Z(3, 8), I(3), 10),
                 lambda: mu.muon_group_norm(Z(3, 8), 2), lambda: mu.muon_group_norm_backward(Z(3, 8), Z(3, 8), 2, None, None, None, Z(3, 2)),
                 lambda: mu.muon_token_logprobs(Z(3, 8), I(3)), lambda: mu.muon_token_logprobs_backward(Z(3, 8), I(3), Z(3, 2), Z(3))):
        with pytest.raises(ValueError, match="must be on cuda"):
            call()


@pytest.mark.parametrize("make,want", [
    (lambda: I(4, 5), (20, 0, 1)), (lambda: I(4, 5)[:, :-1], (4, 5, 1)), (lambda: I(4, 5)[:, 2], (4, 0, 5)), (lambda: I(4, 5)[2], (5, 0, 1)),
    (lambda: I(4, 5).T, (4, 1, 5)), (lambda: I(2, 3, 4)[:, :, :2], (2, 4, 1)), (lambda: I(2, 3, 4)[:, :2], (8, 12, 1)),
    (lambda: I(1).expand(7), (7, 0, 0)), (lambda: I(3, 1).expand(3, 4), (4, 1, 0)), (lambda: I(4, 6)[:, ::2], (12, 0, 2)),
    (lambda: I(5)[:1], (1, 0, 1)), (lambda: I(0), (1, 0, 1)),
])
def test_ids_fold(on_cpu, make, want):
    t = make()
    p, bits, run, stride, step = struct.unpack("@Pi4xqqq", on_cpu.binding._ids(t, "ids", 0))
    assert (run, stride, step) == want and bits == 64 and p == t.data_ptr()
    flat = t.reshape(-1)
    base = torch.arange(t.untyped_storage().nbytes() // 8)
    at = [t.storage_offset() + i // run * stride + i % run * step for i in range(flat.numel())]
    assert torch.equal(base[torch.tensor(at, dtype=torch.long)], base.as_strided(t.shape, t.stride(), t.storage_offset()).reshape(-1))


FAR = (1 << 32) + 8   # in 32 bits: 8


@pytest.mark.parametrize("call", [
    lambda m: m.muon_embedding(torch.empty(FAR, 4, device="meta"), I(3)),
    lambda m: m.muon_embedding(torch.empty(4, FAR, device="meta"), I(1)),
    lambda m: m.muon_embedding_backward(Z(3, 4), I(3), FAR), lambda m: m.muon_embedding_backward(Z(3, 4), I(3), 4 - (1 << 32)),
    lambda m: m.muon_embedding_backward(Z(0, FAR), I(0), 4),
    lambda m: m.muon_embedding_backward_workspace_size(I(3), FAR, 4),
    lambda m: m.muon_group_norm(Z(0, FAR), 1), lambda m: m.muon_group_norm(Z(0, FAR), FAR),
    lambda m: m.muon_group_norm_backward(Z(0, FAR), Z(0, FAR), 2, None, None, None, Z(0, 2)),
    lambda m: m.muon_token_logprobs(Z(0, FAR), I(0)), lambda m: m.muon_token_logprobs(Z(3, 8), I(3), top=FAR),
    lambda m: m.muon_token_logprobs_workspace_size(Z(3, 8), top=FAR),
    lambda m: m.muon_token_logprobs_backward(Z(0, FAR), I(0), Z(0, 2), Z(0)),
])
def test_sizes_past_32_bits_are_not_cut(on_cpu, call, monkeypatch):
    """Refused as themselves, never taken for what their low bits say."""
    B = on_cpu.binding
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(on_cpu.MuonError) as e:
        call(on_cpu)
    assert e.value.status == B.MUON_EUNSUPPORTED
