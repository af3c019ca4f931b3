"""The training example: one checkpoint carried on in 32 and in 8 bits, as a list and as a flat shard."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_training_goes_on_in_8_bits():
    spec = importlib.util.spec_from_file_location("adamw8_training", os.path.join(ROOT, "examples", "adamw8_training.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    found = ex.run(steps=100, say=lambda *_: None)
    assert found["reached"] < 0.5 * found["start"]
    assert found["fp32"] < found["reached"]
    # the moments' 3 bits change the path, not the progress: each run ends within a fifth of the fp32 run's gain
    gain = found["reached"] - found["fp32"]
    for name in ("8 bits, nearest", "8 bits, stochastic", "flat shard"):
        assert found[name] < found["fp32"] + 0.2 * gain + 0.1 * found["fp32"], (name, found)
