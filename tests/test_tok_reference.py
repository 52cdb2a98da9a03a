"""The float64 references of the embedding, the group norm and the token log
probabilities against differences (CPU)."""
import math

import pytest

import tok_reference as ref

torch = pytest.importorskip("torch")

F64 = torch.float64
STEP = 1e-5   # differences of second order: off by STEP^2 times third derivatives of size about 1, and 2^-53 / STEP


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=F64)


def slope(f, x, d):
    return (f(x + STEP * d) - f(x - STEP * d)) / (2 * STEP)


def test_embedding_gradient():
    gen = torch.Generator().manual_seed(1)
    table, dy = normal(gen, 9, 4), normal(gen, 2, 10, 4)
    ids = torch.randint(-2, 12, (2, 10), generator=gen)
    got, size = ref.embedding_grad(dy, ids, 9, -1.5)
    d = normal(gen, 9, 4)
    want = slope(lambda t: (ref.embedding(t, ids, -1.5) * dy).sum(), table, d)
    assert abs((got * d).sum() - want) < 1e-8 and (got.abs() <= size + 1e-12).all()


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("gate,first,act", [(True, True, "silu"), (True, False, "silu"), (False, True, "silu"), (False, True, "none")])
@pytest.mark.parametrize("groups", [1, 3])
def test_group_norm_gradient(groups, gate, first, act, center):
    gen = torch.Generator().manual_seed(2)
    x, dy, w, b = normal(gen, 5, 12), normal(gen, 5, 12), normal(gen, 12), normal(gen, 12)
    z = normal(gen, 5, 12) if gate else None
    f = lambda x, w, b, z: (ref.group_norm(x, groups, w, b, z, first, act, 1e-5, center)[0] * dy).sum()  # noqa: E731
    _, mean, rstd = ref.group_norm(x, groups, w, b, z, first, act, 1e-5, center)
    dx, dz, dw, db = ref.group_norm_grads(dy, x, groups, w, b, mean, rstd, z, first, act)
    for name, at, got in (("x", 0, dx), ("w", 1, dw), ("b", 2, db), ("z", 3, dz)):
        if got is None:
            assert z is None
            continue
        args = [x, w, b, z]
        d = normal(gen, *args[at].shape)
        want = slope(lambda v: f(*args[:at], v, *args[at + 1:]), args[at], d)
        assert abs((got * d).sum() - want) < 1e-6, name


def test_group_norm_of_one_group_is_the_layer_norm():
    import seq_reference
    gen = torch.Generator().manual_seed(3)
    x, w, b = normal(gen, 4, 10), normal(gen, 10), normal(gen, 10)
    for center in (True, False):
        y, _, rstd = ref.group_norm(x, 1, w, b, activation="none", center=center)
        want = seq_reference.norm(x, w, b, center=center)
        assert torch.allclose(y, want[0], atol=1e-12) and torch.allclose(rstd[:, 0], want[2], atol=1e-12)


def test_logprobs_against_torch():
    gen = torch.Generator().manual_seed(4)
    x, ids = 3.0 * normal(gen, 6, 11), torch.tensor([0, 10, -1, 11, 5, 5])
    r = ref.logprobs(x, ids, 0.7, top=4)
    lp = torch.log_softmax(0.7 * x, 1)
    assert torch.allclose(r["entropy"], -(lp.exp() * lp).sum(1), atol=1e-12)
    assert torch.allclose(r["logp"], torch.tensor([lp[0, 0], lp[1, 10], 0, 0, lp[4, 5], lp[5, 5]], dtype=F64), atol=1e-12)
    best = torch.topk(lp, 4, 1)
    assert (r["top_ids"] == best.indices).all() and torch.allclose(r["top_logp"], best.values, atol=1e-12)


def test_logprobs_of_special_rows():
    inf, nan = math.inf, math.nan
    x = torch.tensor([[-inf, -inf, -inf], [-inf, 2.0, -inf], [1.0, nan, 0.0], [1.0, inf, 0.0], [1.0, 1.0, -inf],
                      [torch.finfo(torch.float32).min] * 3], dtype=F64)
    r = ref.logprobs(x, torch.tensor([1, 0, 0, 0, 1, 2]), top=2)
    assert r["logp"][0] == -inf and r["entropy"][0] == 0 and r["top_ids"][0].tolist() == [-1, -1]
    assert r["logp"][1] == -inf and r["entropy"][1] == 0 and r["top_ids"][1].tolist() == [1, -1] and r["top_logp"][1, 0] == 0
    assert torch.isnan(r["logp"][2:4]).all() and torch.isnan(r["entropy"][2:4]).all() and (r["top_ids"][2:4] == -1).all()
    assert abs(r["entropy"][4] - math.log(2)) < 1e-12 and r["top_ids"][4].tolist() == [0, 1]
    assert abs(r["logp"][5] + math.log(3)) < 1e-12 and r["top_ids"][5].tolist() == [0, 1]


def test_logprobs_gradient():
    gen = torch.Generator().manual_seed(5)
    x, ids = 2.0 * normal(gen, 5, 9), torch.tensor([3, -1, 8, 0, 9])
    x[:, 4] = -math.inf
    dl, dh = normal(gen, 5), normal(gen, 5)
    r = ref.logprobs(x, ids, 1.3)
    got, _ = ref.logprobs_grad(x, ids, r["stats"], dl, 1.3, r["entropy"], dh)

    def loss(x):
        s = ref.logprobs(x, ids, 1.3)
        return (s["logp"] * dl).sum() + (s["entropy"] * dh).sum()
    d = normal(gen, 5, 9)
    d[:, 4] = 0.0
    assert abs((got * d).sum() - slope(loss, x, d)) < 1e-7
    assert (got[:, 4] == 0).all()
