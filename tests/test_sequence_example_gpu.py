"""The example policy: training moves the value loss, and the actor's single
steps reach what the learner computes over whole rollouts."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_trains_and_acts():
    assert torch.cuda.is_available(), "the -m gpu tests need a CUDA device"
    spec = importlib.util.spec_from_file_location(
        "sequence_policy", os.path.join(ROOT, "examples", "sequence_policy.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    lines = []
    losses, apart, size = ex.main(updates=20, N=16, T=96, report=lines.append)
    assert losses[-1] < 0.7 * losses[0], losses
    # bfloat16 activations through two mixing layers: a few roundings of 2^-8
    assert apart <= 16 * 2.0 ** -8 * max(size, 0.1), lines
