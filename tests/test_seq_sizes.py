"""Sizes past what the sequence operators' launches and counts hold are
refused (no GPU needed: nothing is enqueued, pointers are made up)."""
import pytest

from test_seq_abi import ADDR, EINVAL, EUNSUPPORTED, args, bwd, fwd, mu, norm, norm_bwd  # noqa: F401

torch = pytest.importorskip("torch")

INT_MAX = 2**31 - 1
AT_ONE = {n: (ADDR[n], 0, 0, 0) for n in ("v", "k", "q", "g")}    # strides that fit any size


@pytest.mark.parametrize("sizes", [
    dict(batch=7_000_000, heads=1, groups=1, P=1, N=1),           # 7e6 walks of 640 work items: past 2^32
    dict(batch=7_000_000, heads=1, groups=1, P=64, N=128),
    dict(batch=1, heads=3_500_000, groups=1, P=65, N=1),          # two blocks of value rows each
    dict(batch=1, heads=1, groups=1, P=INT_MAX, N=1),             # ceil(P / 64) without overflow
    dict(batch=INT_MAX, heads=INT_MAX, groups=1, P=INT_MAX, N=1),
    dict(batch=1 << 30, heads=1 << 30, groups=1 << 30, P=1 << 30, N=1),
], ids=str)
@pytest.mark.parametrize("tokens", [1, 100])
def test_scan_past_a_launch(mu, sizes, tokens):
    a = args(tokens=tokens, **sizes, **AT_ONE)
    L = mu.lib()
    assert L.muon_gated_scan_workspace_size(a) == 0 and L.muon_gated_scan_backward_workspace_size(a) == 0
    assert fwd(mu, a) == EUNSUPPORTED and bwd(mu, a) == EUNSUPPORTED


def test_backward_past_a_launch(mu):
    """Blocks of tokens, which the forward pass walks one after the other."""
    a = args(batch=1000, tokens=1_000_000, heads=1, groups=1, P=1, N=1)
    assert mu.lib().muon_gated_scan_workspace_size(a) > 0
    assert mu.lib().muon_gated_scan_backward_workspace_size(a) == 0 and bwd(mu, a) == EUNSUPPORTED


@pytest.mark.parametrize("sizes", [
    dict(batch=17_000_000, heads=1, groups=1, P=1, N=4), dict(batch=1, heads=9_000_000, groups=1, P=33, N=1),
    dict(batch=1, heads=1, groups=1, P=INT_MAX, N=1), dict(batch=INT_MAX, heads=INT_MAX, groups=1, P=INT_MAX, N=1),
], ids=str)
def test_step_past_a_launch(mu, sizes):
    assert mu.lib().muon_gated_scan_step(args(tokens=1, **sizes, **AT_ONE), ADDR["Y"], ADDR["S"], None) == EUNSUPPORTED


def test_sizes_below_that_are_accepted(mu):
    L = mu.lib()
    assert L.muon_gated_scan_workspace_size(args(batch=6_000_000, tokens=1, heads=1, groups=1, P=64, N=128)) > 0
    assert L.muon_gated_scan_backward_workspace_size(args(batch=1000, tokens=200_000, heads=1, groups=1, P=1, N=1)) > 0


@pytest.mark.parametrize("name", ["v", "k", "q", "g", "b"])
@pytest.mark.parametrize("strides", [(2**62, 1, 1), (1, 2**61, 1), (1, 1, 2**62), (2**63 - 1, 2**63 - 1, 2**63 - 1)], ids=str)
def test_strides_past_any_memory(mu, name, strides):
    """Extents that overflow 64 bits, by which an overlap would go unseen."""
    a = args(**{name: (ADDR["b" if name == "b" else name], *strides)})
    assert fwd(mu, a) == EINVAL and bwd(mu, a) == EINVAL
    one = args(tokens=1, **{name: (ADDR["b" if name == "b" else name], 2**62, 0, 2**62)})
    assert mu.lib().muon_gated_scan_step(one, ADDR["Y"], ADDR["S"], None) == EINVAL


def test_gradient_strides_past_any_memory(mu):
    assert bwd(mu, args(), dY=(ADDR["dY"], 2**62, 256, 64)) == EINVAL


@pytest.mark.parametrize("n", [2**27 + 1, 2**28, 2**30, INT_MAX])
def test_norm_rows_too_long(mu, n):
    """Columns are counted in int, by steps of a workgroup."""
    far = 1 << 50
    assert norm(mu, n=n, ldx=n, ldy=n, rows=1, X=far, Y=2 * far, w=None, b=None) == EUNSUPPORTED
    assert norm_bwd(mu, n=n, ldx=n, lddy=n, lddx=n, rows=1, X=far, dY=2 * far, dX=3 * far, w=None, dw=None, db=None) == EUNSUPPORTED
    assert mu.lib().muon_layer_norm_backward_workspace_size(1, n, 1) == 0
    assert mu.lib().muon_layer_norm_backward_workspace_size(1, 2**27, 1) > 0


@pytest.mark.parametrize("ld", ["ldx", "ldy"])
def test_norm_row_strides_past_any_memory(mu, ld):
    assert norm(mu, **{ld: 2**62}) == EINVAL
    assert norm_bwd(mu, **{"lddx" if ld == "ldy" else ld: 2**62}) == EINVAL and norm_bwd(mu, lddy=2**61) == EINVAL
