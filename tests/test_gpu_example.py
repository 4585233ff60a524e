"""The example that trains with every objective, dropout and the K-FAC step together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy_kfac.py")


def test_example_learns(gpu_lib):
    """The mean reward of a state's ten classes starts near 0.1 and at least doubles; the preference loss falls."""
    spec = importlib.util.spec_from_file_location("policy_kfac", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rewards, losses = example.train(log=lambda line: print(line, flush=True))
    assert rewards[0] < 0.2 and max(rewards[-2:]) > 2 * rewards[0], rewards
    assert sum(losses[-4:]) < 0.8 * sum(losses[:4]), losses
