"""Refusals of the sequence operators, at the C ABI and in the binding: nothing
is enqueued on a bad argument (no GPU needed: pointers are made up and never
read)."""
import ctypes
import os
import struct

import pytest

torch = pytest.importorskip("torch")

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
BIG = 1 << 40


@pytest.fixture(scope="module")
def mu():
    import spectral_optimizer_ssm_amd as mu
    if not os.path.exists(mu.binding.LIB_PATH):
        pytest.fail("libmuon.so is not built: run python -m spectral_optimizer_ssm_amd.build")
    mu.lib()
    return mu


A = 1 << 32            # made-up device addresses, far apart
ADDR = {n: A * (i + 1) for i, n in enumerate(("v", "k", "q", "g", "b", "S0", "Y", "S", "ws", "dY", "dS", "dV", "dK", "dQ",
                                                "dg", "db", "dS0"))}


def args(batch=2, tokens=100, heads=4, groups=2, P=64, N=128, dtype=1, S0=None, **seq):
    """Packed muon_scan_args with contiguous operands at ADDR; seq: other (p, sb, st, sh)."""
    def s(name, h, w):
        return seq.get(name, (ADDR[name], tokens * h * w, h * w, w))
    return struct.pack("@7i4x" + 5 * "Pqqq" + "P", batch, tokens, heads, groups, P, N, dtype, *s("v", heads, P),
                       *s("k", groups, N), *s("q", groups, N), *s("g", heads, 1), *seq.get("b", (0, 0, 0, 0)),
                       ADDR["S0"] if S0 is None else S0)


def fwd(mu, a, Y=ADDR["Y"], S=ADDR["S"], ws=ADDR["ws"], nbytes=BIG):
    return mu.lib().muon_gated_scan(a, Y, S, ws, nbytes, None)


def bwd(mu, a, tokens=100, **kw):
    p = {**{n: ADDR[n] for n in ("dS", "dV", "dK", "dQ", "dg", "db", "dS0", "ws")}, "nbytes": BIG, **kw}
    dy = struct.pack("@Pqqq", *kw.get("dY", (ADDR["dY"], tokens * 256, 256, 64)))
    return mu.lib().muon_gated_scan_backward(a, dy, p["dS"], p["dV"], p["dK"], p["dQ"], p["dg"], p["db"], p["dS0"], p["ws"],
                                             p["nbytes"], None)


def test_workspace_sizes(mu):
    L = mu.lib()
    ok = L.muon_gated_scan_workspace_size(args())
    assert ok > 0 and L.muon_gated_scan_backward_workspace_size(args()) > 2 * 2 * 4 * 64 * 128 * 4
    for bad in (dict(batch=-1), dict(tokens=-1), dict(heads=0), dict(groups=0), dict(heads=3), dict(P=0), dict(N=0),
                dict(N=129), dict(dtype=2)):
        assert L.muon_gated_scan_workspace_size(args(**bad)) == 0, bad
        assert L.muon_gated_scan_backward_workspace_size(args(**bad)) == 0, bad
    assert L.muon_gated_scan_workspace_size(None) == 0
    # few sequences: the time axis is cut, its pieces' states are in the workspace
    assert L.muon_gated_scan_workspace_size(args(batch=1, tokens=16384, heads=24, groups=1)) > 24 * 64 * 128 * 4
    t = lambda *s: torch.empty(*s, dtype=torch.bfloat16)  # noqa: E731
    assert mu.muon_gated_scan_workspace_size(t(2, 100, 4, 64), t(2, 100, 2, 128)) == ok


@pytest.mark.parametrize("bad,expect", [
    (dict(batch=-1), EINVAL), (dict(tokens=-1), EINVAL), (dict(heads=3), EINVAL), (dict(P=0), EINVAL), (dict(N=0), EINVAL),
    (dict(dtype=7), EINVAL), (dict(N=256), EUNSUPPORTED),
    (dict(v=(0, 1, 1, 1)), EINVAL), (dict(k=(0, 1, 1, 1)), EINVAL), (dict(q=(0, 1, 1, 1)), EINVAL),
    (dict(g=(0, 1, 1, 1)), EINVAL), (dict(v=(ADDR["v"] + 1, 25600, 256, 64)), EINVAL),
    (dict(k=(ADDR["k"], -1, 256, 128)), EINVAL), (dict(q=(ADDR["q"], 25600, -256, 128)), EINVAL),
    (dict(g=(ADDR["g"] + 2, 400, 4, 1)), EINVAL), (dict(b=(ADDR["b"] + 2, 400, 4, 1)), EINVAL),
    (dict(b=(ADDR["b"], 400, 4, -1)), EINVAL), (dict(S0=ADDR["S0"] + 2), EINVAL),
], ids=str)
def test_scan_refusals(mu, bad, expect):
    assert fwd(mu, args(**bad)) == expect
    assert bwd(mu, args(**bad)) == expect
    one = {k: v for k, v in bad.items()}
    one.setdefault("tokens", 1)
    assert mu.lib().muon_gated_scan_step(args(**one), ADDR["Y"], ADDR["S"], None) == expect


def test_scan_output_refusals(mu):
    a = args()
    assert fwd(mu, None) == EINVAL
    assert fwd(mu, a, Y=None) == EINVAL and fwd(mu, a, Y=ADDR["Y"] + 1) == EINVAL and fwd(mu, a, S=ADDR["S"] + 2) == EINVAL
    assert fwd(mu, a, ws=None) == EWORKSPACE and fwd(mu, a, nbytes=0) == EWORKSPACE and fwd(mu, a, ws=ADDR["ws"] + 4) == EWORKSPACE
    # overlaps: outputs with inputs, with the workspace and with each other
    for o in ("v", "k", "q", "g", "S0"):
        assert fwd(mu, a, Y=ADDR[o] + 64) == EINVAL and fwd(mu, a, S=ADDR[o] + 64) == EINVAL and fwd(mu, a, ws=ADDR[o]) == EINVAL, o
    assert fwd(mu, a, Y=ADDR["S"]) == EINVAL and fwd(mu, a, ws=ADDR["Y"]) == EINVAL
    for o in ("dV", "dK", "dQ", "dg"):
        assert bwd(mu, a, **{o: None}) == EINVAL, o
        assert bwd(mu, a, **{o: ADDR[o] + 1}) == EINVAL, o
        assert bwd(mu, a, **{o: ADDR["q"] + 64}) == EINVAL, o
        assert bwd(mu, a, **{o: ADDR["dS"]}) == EINVAL, o
    for o in ("db", "dS0", "dS"):
        assert bwd(mu, a, **{o: ADDR[o] + 2}) == EINVAL, o
    assert bwd(mu, a, dY=(0, 1, 1, 1)) == EINVAL and bwd(mu, a, dY=(ADDR["dY"], 25600, 256, -64)) == EINVAL
    assert bwd(mu, a, ws=None) == EWORKSPACE and bwd(mu, a, nbytes=100) == EWORKSPACE
    assert bwd(mu, a, dV=ADDR["dK"]) == EINVAL
    L = mu.lib()
    one = args(tokens=1)
    assert L.muon_gated_scan_step(args(tokens=2), ADDR["Y"], ADDR["S"], None) == EINVAL
    assert L.muon_gated_scan_step(args(tokens=1, S0=0), ADDR["Y"], ADDR["S"], None) == EINVAL
    assert L.muon_gated_scan_step(one, ADDR["Y"], None, None) == EINVAL
    assert L.muon_gated_scan_step(one, ADDR["Y"], ADDR["S"] + 4, None) == EINVAL    # N % 4 == 0: 16-byte rows
    assert L.muon_gated_scan_step(one, ADDR["Y"], ADDR["S0"] + 16, None) == EINVAL  # neither in place nor apart
    assert L.muon_gated_scan_step(one, ADDR["S"], ADDR["S"], None) == EINVAL
    # nothing to do
    assert fwd(mu, args(batch=0), Y=None, S=None, ws=None, nbytes=0) == 0


def norm(mu, X=ADDR["v"], ldx=768, dtype=1, rows=10, n=768, w=ADDR["k"], b=ADDR["q"], eps=1e-5, center=1, Y=ADDR["Y"], ldy=768,
         mean=ADDR["dg"], rstd=ADDR["db"]):
    return mu.lib().muon_layer_norm(X, ldx, dtype, rows, n, w, b, eps, center, Y, ldy, mean, rstd, None)


def norm_bwd(mu, dY=ADDR["dY"], lddy=768, X=ADDR["v"], ldx=768, dtype=1, rows=10, n=768, w=ADDR["k"], mean=ADDR["g"], rstd=ADDR["b"],
             dX=ADDR["dV"], lddx=768, dw=ADDR["dK"], db=ADDR["dQ"], ws=ADDR["ws"], nbytes=BIG):
    return mu.lib().muon_layer_norm_backward(dY, lddy, X, ldx, dtype, rows, n, w, mean, rstd, dX, lddx, dw, db, ws, nbytes, None)


@pytest.mark.parametrize("bad,expect", [
    (dict(dtype=3), EINVAL), (dict(rows=-1), EINVAL), (dict(n=0), EINVAL), (dict(rows=1 << 31), EUNSUPPORTED),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(center=2), EINVAL), (dict(ldx=767), EINVAL),
    (dict(ldy=700), EINVAL), (dict(X=None), EINVAL), (dict(Y=None), EINVAL), (dict(X=ADDR["v"] + 1), EINVAL),
    (dict(Y=ADDR["Y"] + 1), EINVAL), (dict(w=ADDR["k"] + 2), EINVAL), (dict(b=ADDR["q"] + 1), EINVAL),
    (dict(mean=ADDR["dg"] + 2), EINVAL), (dict(rstd=ADDR["db"] + 2), EINVAL), (dict(Y=ADDR["v"]), EINVAL),
    (dict(Y=ADDR["v"] + 1536), EINVAL), (dict(mean=ADDR["k"]), EINVAL), (dict(mean=ADDR["db"]), EINVAL),
], ids=str)
def test_norm_refusals(mu, bad, expect):
    assert norm(mu, **bad) == expect


@pytest.mark.parametrize("bad,expect", [
    (dict(dtype=3), EINVAL), (dict(rows=-1), EINVAL), (dict(n=0), EINVAL), (dict(lddy=1), EINVAL), (dict(ldx=1), EINVAL),
    (dict(lddx=1), EINVAL), (dict(dY=None), EINVAL), (dict(X=None), EINVAL), (dict(dX=None), EINVAL), (dict(rstd=None), EINVAL),
    (dict(dX=ADDR["dV"] + 1), EINVAL), (dict(dw=ADDR["dK"] + 2), EINVAL), (dict(mean=ADDR["g"] + 1), EINVAL),
    (dict(ws=None), EWORKSPACE), (dict(nbytes=16), EWORKSPACE), (dict(ws=ADDR["ws"] + 8), EWORKSPACE),
    (dict(dX=ADDR["v"]), EINVAL), (dict(dX=ADDR["dY"] + 64), EINVAL), (dict(dw=ADDR["dQ"]), EINVAL), (dict(dw=ADDR["k"]), EINVAL),
], ids=str)
def test_norm_backward_refusals(mu, bad, expect):
    assert norm_bwd(mu, **bad) == expect


def test_norm_nothing_to_do(mu):
    assert norm(mu, rows=0, X=None, Y=None) == 0
    assert norm_bwd(mu, rows=0, dY=None, X=None, dX=None, rstd=None, dw=None, db=None, ws=None, nbytes=0) == 0
    L = mu.lib()
    assert L.muon_layer_norm_backward_workspace_size(10, 0, 1) == 0 and L.muon_layer_norm_backward_workspace_size(10, 8, 5) == 0
    assert L.muon_layer_norm_backward_workspace_size(10, 768, 1) >= 2 * 768 * 4


# ---------------------------------------------------------------------------
# the binding's own checks (tensors on the CPU: the device is checked last)
# ---------------------------------------------------------------------------
def tensors(B=2, T=5, H=4, G=2, P=6, N=8, dt=torch.bfloat16):
    return dict(V=torch.zeros(B, T, H, P, dtype=dt), K=torch.zeros(B, T, G, N, dtype=dt), Q=torch.zeros(B, T, G, N, dtype=dt),
                log_decay=torch.zeros(B, T, H), gate=torch.zeros(B, T, H), S0=torch.zeros(B, H, P, N))


@pytest.mark.parametrize("change,error", [
    (dict(V=torch.zeros(2, 5, 24)), ValueError), (dict(K=torch.zeros(2, 5, 2, 9, dtype=torch.bfloat16)), ValueError),
    (dict(Q=torch.zeros(2, 4, 2, 8, dtype=torch.bfloat16)), ValueError),
    (dict(K=torch.zeros(2, 5, 3, 8, dtype=torch.bfloat16), Q=torch.zeros(2, 5, 3, 8, dtype=torch.bfloat16)), ValueError),
    (dict(V=torch.zeros(2, 5, 4, 6, dtype=torch.float16)), TypeError), (dict(K=torch.zeros(2, 5, 2, 8)), TypeError),
    (dict(Q=torch.zeros(2, 5, 2, 8)), TypeError), (dict(log_decay=torch.zeros(2, 5, 3)), ValueError),
    (dict(log_decay=torch.zeros(2, 5, 4, dtype=torch.float64)), TypeError), (dict(gate=torch.zeros(2, 5)), ValueError),
    (dict(gate=torch.zeros(2, 5, 4, dtype=torch.bfloat16)), TypeError), (dict(S0=torch.zeros(2, 4, 8, 6)), ValueError),
    (dict(S0=torch.zeros(2, 4, 8, 6).transpose(2, 3)), ValueError), (dict(S0=torch.zeros(2, 4, 6, 8).double()), TypeError),
    (dict(V=torch.zeros(2, 5, 6, 4, dtype=torch.bfloat16).transpose(2, 3)), ValueError),
    (dict(), ValueError),   # on the CPU
], ids=lambda x: "+".join(x) if isinstance(x, dict) else x.__name__)
def test_binding_refuses_scan_arguments(mu, monkeypatch, change, error):
    B = mu.binding
    monkeypatch.setattr(B, "_device_index", lambda: 0)
    if B.torch is None:
        B._load_torch()
    if change:   # everything but the change is taken to be where it should
        monkeypatch.setattr(B, "_where", lambda t, name, index: None)
    x = {**tensors(), **change}
    with pytest.raises(error):
        mu.muon_gated_scan(x["V"], x["K"], x["Q"], x["log_decay"], gate=x["gate"], S0=x["S0"], Y=torch.zeros(1))
    with pytest.raises(error):
        mu.muon_gated_scan_backward(x["V"], x["K"], x["Q"], x["log_decay"], tensors()["V"], gate=x["gate"], S0=x["S0"], dV=torch.zeros(1))


@pytest.mark.parametrize("kw,error", [
    (dict(weight=torch.zeros(7)), ValueError), (dict(bias=torch.zeros(2, 4)), ValueError),
    (dict(weight=torch.zeros(8, dtype=torch.bfloat16)), TypeError), (dict(X=torch.zeros(3, 8, dtype=torch.float16)), TypeError),
    (dict(X=torch.zeros(8, 3).T), ValueError), (dict(X=torch.zeros(2, 4, 3, 8)[:, ::2, ::2]), ValueError),
    (dict(Y=torch.zeros(3, 9)), ValueError), (dict(Y=torch.zeros(3, 8, dtype=torch.bfloat16)), TypeError), (dict(), ValueError),
], ids=lambda x: "+".join(x) if isinstance(x, dict) else x.__name__)
def test_binding_refuses_norm_arguments(mu, monkeypatch, kw, error):
    B = mu.binding
    monkeypatch.setattr(B, "_device_index", lambda: 0)
    if B.torch is None:
        B._load_torch()
    if kw:
        monkeypatch.setattr(B, "_where", lambda t, name, index: None)
    with pytest.raises(error):
        mu.muon_layer_norm(kw.pop("X", torch.zeros(3, 8)), **kw)


def test_scan_args_match_the_header(mu, tmp_path):
    """The packed record is muon_scan_args as a C compiler lays it out."""
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "muon.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu %zu %zu %zu", sizeof(muon_scan_args), offsetof(muon_scan_args, dtype),'
                   ' offsetof(muon_scan_args, v), offsetof(muon_scan_args, q), offsetof(muon_scan_args, gate),'
                   ' offsetof(muon_scan_args, S0), sizeof(muon_seq));return 0;}\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "t")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "t")], capture_output=True, text=True).stdout.split()]
    assert got == [mu.binding._SCAN_ARGS.size, 24, 32, 32 + 64, 32 + 128, 32 + 160, mu.binding._SEQ.size]
