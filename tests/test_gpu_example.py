"""The example that runs the operators together as a training step."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "training_step.py")


def test_training_step_learns_and_repeats(dev):
    spec = importlib.util.spec_from_file_location("training_step", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=30)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0]
    assert example.train(steps=30) == losses
