"""A state that is not finite ends with its sequence: results of sequences that
start after it are bit for bit those without it."""
import math

import pytest

from test_gpu_gated_scan import BF16, F32, _announce, backward, forward, inputs, mu  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BAD = [math.nan, math.inf, -math.inf]
both = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


def equal(got, want, where=slice(None)):
    for a, b in zip(got, want):
        if a is not None:
            assert torch.isfinite(b[:, where]).all() and torch.equal(a[:, where], b[:, where])


@both
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("tokens", [1, 150, 1400])
def test_initial_state_before_a_start(mu, tokens, bad, dtype):
    """A slot that some other sequence has left, or memory that was never written."""
    x = inputs(1, tokens, 2, 2, 64, 128, dtype, seed=71)
    x["g"][:, 0] = -math.inf
    want, grads = forward(mu, x), backward(mu, x)
    x["S0"][:, 0] = bad
    x["S0"][:, 1, 3, 5] = bad
    equal(forward(mu, x), want)
    equal(backward(mu, x), grads)


@both
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("batch", [2, 400])
def test_step_that_starts_a_sequence(mu, batch, bad, dtype):
    x = inputs(batch, 1, 2, 1, 64, 72, dtype, seed=72)
    x["g"][::2] = -math.inf
    one = [x[n][:, 0].cuda() for n in ("v", "k", "q", "g")]
    S = x["S0"].cuda()
    want = mu.muon_gated_scan_step(*one, S, gate=x["b"][:, 0].cuda(), S_out=torch.empty_like(S))
    S[::2] = bad
    got = mu.muon_gated_scan_step(*one, S, gate=x["b"][:, 0].cuda())
    equal(got, want)


@both
@pytest.mark.parametrize("tokens", [400, 1500])
def test_sequences_after_one_that_is_not_finite(mu, tokens, dtype):
    """One packed sequence has a NaN among its values: those that start in later
    blocks of tokens are not reached, forward and back."""
    x = inputs(1, tokens, 2, 2, 64, 128, dtype, seed=73, state=False)
    x["g"][:, [200, 256, 330]] = -math.inf
    want, grads = forward(mu, x), backward(mu, x)
    z = {**x, "v": x["v"].clone()}
    z["v"][:, 50, 0, 7] = math.nan
    y, S = forward(mu, z)
    assert torch.isnan(y[:, 60]).any()
    equal([y], want[:1], slice(256, None))
    equal([S], want[1:])
    equal(backward(mu, z)[:5], grads[:5], slice(256, None))
    z = {**x, "dy": x["dy"].clone()}
    z["dy"][:, 350, 1, 2] = math.inf
    got = backward(mu, z)
    assert not torch.isfinite(got[0][:, 340]).all()
    equal(got[:5], grads[:5], slice(0, 256))
