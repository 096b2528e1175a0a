"""The example's sampler in FP8: its view after every patch is the codes of the served weights, its logits their product."""
import os
import sys

import numpy as np
import pytest
import torch

import rl_post_trainer_gb300 as pulse
import serving_ref as ref
from test_gpu_fp8 import check_product, host

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_view_and_logits_follow_the_patches():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    import rollout_and_step as example
    gen = torch.Generator(device="cuda").manual_seed(2)
    trainer = example.Trainer(32, gen)
    sampler = example.Fp8Sampler(trainer)
    tokens = torch.randint(0, example.VOCAB, (example.SEQUENCES,), generator=gen, device="cuda", dtype=torch.int32)
    before = None
    for step in range(3):
        if step:  # a step of the trainer's, and its patch
            for g in trainer.grads:
                g.normal_(generator=gen)
            _, clip = trainer.adam.grad_norm(1.0)
            trainer.adam.step(step, 0.05, grad_scale=clip, seed=1)
            sampler.apply(trainer.encode())
            sampler.renew()
        codes, scales = ref.quantize(host(sampler.weights[1]), pulse.FP8_BLOCK)
        np.testing.assert_array_equal(host(sampler.view[0]), codes)
        np.testing.assert_array_equal(host(sampler.view[1]), scales)
        assert before is None or (codes != before).any()
        before = codes
        x, x_scales = ref.quantize(host(sampler.weights[0][tokens.long()]), 1)
        logits = sampler.logits(tokens)
        check_product(x, x_scales, codes, scales, logits, torch.bfloat16)
    assert pulse.get_error() == 0
