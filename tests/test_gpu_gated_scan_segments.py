"""Rows so long, and so few, that the time axis is cut into segments, in both
directions: forward from 8 chunks of 64 tokens on, backward from 20, where fewer
than 39 heads and blocks of value rows walk.  That a case is cut is read off its
workspace."""
import math

import pytest

import seq_reference as ref
from test_gpu_gated_scan import BF16, F32, F32_TOL, _announce, backward, check_backward, check_forward, forward, inputs, mu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def segments(mu, x):
    """Segments of the forward and of the backward walk (heads do not share keys: no other parts in the workspace)."""
    B, T, H, P = x["v"].shape
    assert x["k"].shape[2] == H
    rows = B * H * -(-P // 64)
    tile = 64 * (64 if x["k"].shape[3] <= 64 else 128) * 4
    blocks = -(-T // (128 if x["v"].dtype == BF16 else 64))
    fwd = mu.muon_gated_scan_workspace_size(x["v"], x["k"]) // (rows * tile)
    bwd = (mu.muon_gated_scan_workspace_size(x["v"], x["k"], backward=True) - 2 * rows * blocks * tile) // (2 * rows * tile)
    return fwd, bwd


SHAPES = [  # B, T, H, G, P, N
    (1, 1300, 1, 1, 64, 128),
    (1, 3000, 1, 1, 64, 128),
    (2, 2100, 2, 2, 64, 64),
    (1, 1281, 1, 1, 130, 100),     # three blocks of value rows, a last chunk of one token
    (1, 1400, 2, 2, 17, 33),       # read element by element
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_segments(mu, shape, dtype):
    x = inputs(*shape, dtype, seed=51, decay=0.02)
    fwd, bwd = segments(mu, x)
    print(f"[case] {fwd} and {bwd} segments", flush=True)
    assert fwd >= 4 and bwd >= 5
    check_forward(mu, x)
    check_backward(mu, x)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("where", ["edges", "beside", "few", "many"])
def test_resets_across_segments(mu, where, dtype):
    """Sequences that start at the chunks' edges (so at the segments' too), just
    before and after them, seldom (segments without any), and at every other token."""
    shape = (1, 2000, 2, 2, 64, 128)
    x = inputs(*shape, dtype, seed=52, decay=0.02, resets=0.5 if where == "many" else 0.0)
    gen = torch.Generator().manual_seed(53)
    if where == "edges":
        x["g"][:, ::64] = -math.inf
    elif where == "beside":
        at = 64 * torch.arange(1, 31) + torch.randint(-1, 2, (30,), generator=gen)
        x["g"][:, at] = -math.inf
    elif where == "few":
        x["g"][:, [700, 1407]] = -math.inf
    assert min(segments(mu, x)) >= 5
    check_forward(mu, x)
    check_backward(mu, x)


@pytest.mark.parametrize("gate,state", [(False, False), (False, True), (True, False)])
def test_segments_without_gate_or_states(mu, gate, state):
    x = inputs(1, 1500, 3, 3, 64, 128, BF16, seed=54, decay=0.01, gate=gate, state=state)
    assert min(segments(mu, x)) >= 5
    check_forward(mu, x)
    check_backward(mu, x)


def test_shared_keys_in_segments(mu):
    """Heads that share keys, split over workgroups, in rows that are cut."""
    x = inputs(1, 1700, 6, 1, 64, 128, BF16, seed=55, decay=0.02, resets=0.002)
    check_forward(mu, x)
    check_backward(mu, x)


def test_segments_are_the_sequence_in_calls(mu):
    """A row that is cut, and the same in two calls that carry the state."""
    x = inputs(1, 1600, 2, 2, 64, 128, F32, seed=56, decay=0.005)
    assert segments(mu, x)[0] >= 4
    y, S = forward(mu, x)
    cut = lambda s: {n: t if n in ("S0", "dS") else t[:, s].contiguous() for n, t in x.items()}  # noqa: E731
    y1, S1 = forward(mu, cut(slice(0, 777)))
    y2, S2 = forward(mu, {**cut(slice(777, None)), "S0": S1.cpu()})
    assert ref.rel(torch.cat([y1, y2], 1), y.cpu()) <= F32_TOL and ref.rel(S2, S.cpu()) <= F32_TOL
