"""The float64 references of the sequence operators: gradients against central
differences, and known values (no GPU)."""
import math

import pytest

torch = pytest.importorskip("torch")

import seq_reference as ref  # noqa: E402

H = 1e-5          # step of the central differences: error ~ H^2 + 2^-52 / H ~ 1e-10 relative
DIFF_TOL = 1e-7


def draw(*shape, gen):
    return torch.randn(*shape, generator=gen, dtype=torch.float64)


def test_scan_known_values():
    """Decay 1, gate 1: S is the plain sum; a reset drops everything before it."""
    gen = torch.Generator().manual_seed(1)
    v, k, q = draw(1, 5, 1, 3, gen=gen), draw(1, 5, 1, 4, gen=gen), draw(1, 5, 1, 4, gen=gen)
    g = torch.zeros(1, 5, 1, dtype=torch.float64)
    y, S, _ = ref.scan(v, k, q, g)
    assert torch.allclose(S[0, 0], v[0, :, 0].T @ k[0, :, 0])
    g[0, 3, 0] = -math.inf
    y, S, _ = ref.scan(v, k, q, g, S0=torch.full((1, 1, 3, 4), 7.0))
    assert torch.allclose(S[0, 0], v[0, 3:, 0].T @ k[0, 3:, 0])
    assert torch.allclose(y[0, 3, 0], v[0, 3, 0] * (k[0, 3, 0] @ q[0, 3, 0]))


@pytest.mark.parametrize("seed", range(3))
def test_scan_gradients_are_differences(seed):
    gen = torch.Generator().manual_seed(seed)
    B, T, Hh, G, P, N = 2, 7, 4, 2, 3, 5
    x = {"v": draw(B, T, Hh, P, gen=gen), "k": draw(B, T, G, N, gen=gen), "q": draw(B, T, G, N, gen=gen),
         "g": -draw(B, T, Hh, gen=gen).abs(), "b": draw(B, T, Hh, gen=gen), "S0": draw(B, Hh, P, N, gen=gen)}
    dy, dS = draw(B, T, Hh, P, gen=gen), draw(B, Hh, P, N, gen=gen)

    def loss(**z):
        y, S, _ = ref.scan(**z)
        return float((y * dy).sum() + (S * dS).sum())

    grads = dict(zip(("v", "k", "q", "g", "b", "S0"), ref.scan_grads(**x, dy=dy, dS=dS)))
    for name in x:
        d = draw(*x[name].shape, gen=gen)
        diff = (loss(**{**x, name: x[name] + H * d}) - loss(**{**x, name: x[name] - H * d})) / (2 * H)
        got = float((grads[name] * d).sum())
        assert abs(got - diff) <= DIFF_TOL * float(grads[name].norm() * d.norm()), name


@pytest.mark.parametrize("center", [True, False])
def test_norm_gradients_are_differences(center):
    gen = torch.Generator().manual_seed(5)
    x, w, bias, dy = draw(4, 9, gen=gen), draw(9, gen=gen), draw(9, gen=gen), draw(4, 9, gen=gen)

    def loss(x, w, bias):
        return float((ref.norm(x, w, bias, center=center)[0] * dy).sum())

    _, mu, r = ref.norm(x, w, bias, center=center)
    grads = ref.norm_grads(dy, x, w, mu, r, center)
    args = [x, w, bias]
    for i, g in enumerate(grads):
        d = draw(*args[i].shape, gen=gen)
        at = lambda s: [a + s * d if j == i else a for j, a in enumerate(args)]  # noqa: E731
        diff = (loss(*at(H)) - loss(*at(-H))) / (2 * H)
        assert abs(float((g * d).sum()) - diff) <= DIFF_TOL * float(g.norm() * d.norm())
