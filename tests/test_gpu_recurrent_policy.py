"""The example policy: acting step by step and scoring the same window at once give the same
outputs, and training on the library's advantages learns to recall."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("recurrent_policy",
                                                  os.path.join(ROOT, "examples", "recurrent_policy.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_learns_and_agrees(example):
    history, drift = example.main(["--updates", "60", "--quiet"])
    # one pass steps, the other sums in chunks: both fp32, outputs of order 1 to 10
    assert drift <= 1e-3, drift
    assert sum(history[-5:]) / 5 >= 0.5, history  # twice the chance of 0.25
