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


def test_sampler_and_trainer_shape_alike():
    """Equal logits get equal bits from both plans: no setting is dropped on one side."""
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    import rollout_and_step as example
    gen = torch.Generator(device="cuda").manual_seed(5)
    n, prompt, length, vocab = example.SEQUENCES, example.PROMPT, example.LENGTH, example.VOCAB
    # few different tokens, so that histories repeat them
    tokens = torch.randint(0, 40, (n, prompt + length), generator=gen, device="cuda", dtype=torch.int32)
    decode, train, split, end = example.plans(tokens)
    raw = torch.randn(n, length, vocab, generator=gen, device="cuda").to(torch.bfloat16)
    shaped = train.shape(raw.view(-1, vocab), out_dtype=torch.float32).view(n, length, vocab)
    d = torch.randn(n, length, vocab, generator=gen, device="cuda")
    back = train.backward(d.view(-1, vocab), logits=raw.view(-1, vocab)).view(n, length, vocab)
    for t in range(length):
        end.copy_(split + t)
        assert torch.equal(decode.shape(raw[:, t], out_dtype=torch.float32), shaped[:, t])
        assert torch.equal(decode.backward(d[:, t], logits=raw[:, t]), back[:, t])
    assert not torch.equal(shaped[:, 0], shaped[:, -1])
