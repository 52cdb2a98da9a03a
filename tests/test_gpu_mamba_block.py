"""The example block: the new operators, Muon and AdamW trained together, and
the trained block decoded token by token."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("mamba_block", os.path.join(ROOT, "examples", "mamba_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_block_trains_and_decodes(example):
    losses, block = example.train(steps=30, batch=2, tokens=150)
    print(f"[case] loss {losses[0]:.4f} -> {losses[-1]:.4f}", flush=True)
    # two independent blocks differ by about the size of what they add; training has to take a good part of it away
    assert all(l == l for l in losses) and losses[-1] < 0.7 * losses[0], losses
    # both ways round the same bfloat16 products at other places: a few times 2^-8 of an output's size
    assert example.decode_difference(block) < 0.1
