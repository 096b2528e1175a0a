"""The example loop: rollout, shaped policy gradient, clipped step, patch, apply."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("state_bits", [32, 8])
def test_rollout_and_step(state_bits):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    import rollout_and_step
    rewards, apart = rollout_and_step.run(iterations=12, state_bits=state_bits)
    # a fifth of the tokens is rewarded by chance; the gradient has to be of use
    assert sum(rewards[-3:]) / 3 > sum(rewards[:3]) / 3 + 0.1
    # BF16 logits of the same weights, from two matrix products of different heights: rarely a last bit apart
    assert apart < 0.2
