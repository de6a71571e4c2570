"""The example that runs the training operators with the compressor (GPU): it learns, and its
single-token form continues what its sequence form computed."""
import math
import os
import sys

import pytest
import torch

from _gpu import ensure_built

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_the_example_learns(state_bits):
    import recurrent_lm
    _, losses = recurrent_lm.train(steps=120, learners=2, state_bits=state_bits)
    least = recurrent_lm.Text().entropy()
    assert abs(losses[0] - math.log(64)) < 0.3  # an untrained model knows nothing
    assert sum(losses[-10:]) / 10 < least + 0.5 * (losses[0] - least), (losses[::10], least)


def test_one_token_at_a_time_is_the_sequence():
    import recurrent_lm
    model = recurrent_lm.Model(seed=3)
    tokens = recurrent_lm.Text().batch(5, 40)
    with torch.no_grad():
        whole = model.logits(tokens)[:, -1]
    _, last = model.generate(tokens, 1)
    assert (whole - last).abs().max() < 1e-3 * whole.abs().max()
