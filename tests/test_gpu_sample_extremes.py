"""Sampling at the ends of what temperatures and logits can be, against the definition in float64."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_gpu_sample import call, check, logits

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
LEAST = 2.0 ** -127
CUTS = [dict(), dict(top_k=7), dict(top_p=0.6), dict(top_p=0.999), dict(min_p=0.3), dict(min_p=1.0), dict(min_p=1.5), dict(top_k=300, top_p=0.9, min_p=0.01)]


def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [5, 1000, 40000])
@pytest.mark.parametrize("temperature", [1e-45, 1e-40, 4e-39, 1e-38, LEAST, 1e-37, 1e-30, 1e-12, 1e-5, 1e5, 1e12, 1e30])
def test_logits_of_the_temperatures_size(vocab, temperature, dtype):
    """Logits some temperatures apart; temperatures below 2^-127 count as that."""
    _cuda()
    counts = max(float(np.float32(temperature)), LEAST)
    x = (logits(4, vocab, F32, vocab).double() * counts).to(dtype)
    for k, s in enumerate(CUTS):
        u = np.random.default_rng(k).random(4).astype(np.float32)
        got = call(x, u, temperature=temperature, **s)
        check(x, u, got, temperature=counts, **s)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [5, 1000, 40000])
def test_infinite_temperature(vocab, dtype):
    """All tokens alike, so that only top-k tells them apart; logits in the order that the ranks have."""
    _cuda()
    x = logits(4, vocab, dtype, vocab)
    for k, s in enumerate(CUTS):
        u = np.random.default_rng(k).random(4).astype(np.float32)
        tokens, logprobs = call(x, u, temperature=np.inf, **s)
        if s.get("min_p", 0) >= 1:
            top = x.float().amax(1, keepdim=True)
            assert (x.float().gather(1, torch.from_numpy(tokens).long()[:, None]) == top).all()
        else:
            for r, row in enumerate(x.float().numpy()):
                order = np.argsort(-row, kind="stable")[:s.get("top_k") or vocab]
                n = min(order.size, int(np.ceil(float(np.float32(s.get("top_p", 1.0))) * order.size)))
                kept = np.sort(order[:max(1, n)])
                assert tokens[r] == kept[int(float(u[r]) * kept.size)], (s, r)
        np.testing.assert_allclose(logprobs, -np.log(vocab), rtol=0, atol=2.0 ** -17)


def test_min_p_of_one():
    """The tokens of the largest logit, and no others, however near they are (a weight next to 1 is 1 in float64)."""
    _cuda()
    x = torch.zeros(64, 3000)
    x[:, [5, 700, 2999]] = 1.0
    x[:, 9] = float(np.nextafter(np.float32(1), np.float32(0)))
    u = np.random.default_rng(0).random(64).astype(np.float32)
    for p in (1.0, 1.5, np.inf):
        for t in (1.0, 1e30):
            tokens, _ = call(x, u, temperature=t, min_p=p)
            np.testing.assert_array_equal(tokens, np.array([5, 700, 2999])[(u * np.float64(3)).astype(int)])
