"""bfloat16 results of the gated scan are rounded once, whatever the length of
the sequences and wherever they start in a packed row.

A result y + d, |d| <= delta, rounds to within |round(y) - y| + 2 delta of y.
Operands that are kept in two bfloat16 pieces are within 2^-16 of their
value, so terms of five times the result's size add 2 * 5 * 2^-16 = 1.5e-4,
under a tenth of the 1.7e-3 that rounding itself leaves: 1.1 times the error of
the rounded float64 result is allowed."""
import math

import pytest

import seq_reference as ref
from test_gpu_gated_scan import _announce, backward, forward, inputs, mu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16
RATIO = 1.1
SHAPES = [  # B, T, H, G, P, N
    (1, 65, 4, 2, 64, 128),
    (2, 130, 4, 2, 64, 128),
    (2, 300, 3, 1, 80, 72),
    (3, 200, 2, 1, 17, 5),
    (1, 500, 6, 1, 64, 64),
    (1, 1500, 2, 1, 64, 128),      # several segments of the time axis
]


def _rounded_once(mu, x, first=None):
    """Errors of y, dv, dk and dq against those of the rounded float64 results
    (first: over the first tokens of the rows only)."""
    want = {"y": ref.scan(x["v"], x["k"], x["q"], x["g"], x["b"], x["S0"])[0]}
    want.update(zip(("dv", "dk", "dq"), ref.scan_grads(x["v"], x["k"], x["q"], x["g"], x["dy"], x["b"], x["S0"], x["dS"])))
    got = {"y": forward(mu, x)[0]}
    got.update(zip(("dv", "dk", "dq"), backward(mu, x)))
    for name, w in want.items():
        a, w = got[name][:, :first], w[:, :first]
        once, err = ref.rel(w.to(BF16), w), ref.rel(a, w)
        print(f"[parity] {name} {err:.2e} rounding {once:.2e}", flush=True)
        assert err <= RATIO * once, (name, err, once)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sequences_of_many_chunks(mu, shape):
    _rounded_once(mu, inputs(*shape, BF16, seed=21))


@pytest.mark.parametrize("shape", SHAPES[:2], ids=str)
def test_first_tokens(mu, shape):
    """Few terms, of which a rounded one would move a whole row."""
    _rounded_once(mu, inputs(*shape, BF16, seed=22, state=False), first=4)


@pytest.mark.parametrize("resets", [0.02, 0.5, 1.0])
def test_packed_sequences(mu, resets):
    _rounded_once(mu, inputs(2, 260, 4, 1, 64, 128, BF16, seed=23, resets=resets))


def test_packed_is_as_alone(mu):
    """A sequence of 40 tokens inside a row of 200, and alone: the same but for
    the last rounding."""
    x = inputs(1, 200, 4, 1, 64, 128, BF16, seed=24, state=False)
    x["g"][:, 90] = x["g"][:, 130] = -math.inf
    alone = {n: None if t is None else t[:, 90:130].contiguous() for n, t in x.items()}
    w = ref.scan(alone["v"], alone["k"], alone["q"], alone["g"], alone["b"])[0]
    once = ref.rel(w.to(BF16), w)
    for y in (forward(mu, x)[0][:, 90:130], forward(mu, alone)[0]):
        assert ref.rel(y, w) <= RATIO * once
