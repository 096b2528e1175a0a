"""Codes of blocks with small scales: quotients on and next to the borders between two codes, for scales of all 24 bits,
where what a quotient leaves over nears the smallest FP32 numbers."""
import numpy as np
import pytest
import torch

import rl_post_trainer_gb300 as pulse
import serving_ref as ref

pytestmark = pytest.mark.gpu

BORDERS = np.unique(np.abs(ref.e4m3_value(np.arange(127, dtype=np.uint8))))
BORDERS = (BORDERS[1:] + BORDERS[:-1]) / 2  # 126 of them


def blocks(exponent, dtype, seed):
    """Blocks whose largest is 448 times a scale of that exponent, the others the borders times it and their neighbours."""
    g = np.random.default_rng(seed)
    fraction = 1 + g.integers(0, 1 << 23, 120) / 2.0 ** 23
    fraction[:60] = (1 + np.arange(60) // 13 * 13 / 64.0)[:60]  # of few bits, whose ties BF16 inputs meet
    amax = torch.from_numpy((fraction * 448.0 * 2.0 ** exponent).astype(np.float32)).to(dtype).float().numpy()
    scale = np.maximum(amax / np.float32(448), np.float32(2.0 ** -126)).astype(np.float64)
    x = np.zeros((3, amax.size, 128), np.float32)
    for k, step in enumerate((-1, 0, 1)):
        at = torch.from_numpy((scale[:, None] * BORDERS).astype(np.float32)).to(dtype)
        bits = at.view(torch.int32 if dtype == torch.float32 else torch.int16)
        at = (bits + step).clamp_(min=0).view(dtype).float().numpy()
        x[k, :, 1:127] = np.minimum(at, amax[:, None]) * np.where(g.random(at.shape) < 0.5, -1, 1)
    x[:, :, 0] = amax
    return torch.from_numpy(x.reshape(-1, 128)).to(dtype)


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("exponent", list(range(-127, -86)) + [-50, 0, 100, 118])
def test_small_scales(exponent, dtype, tall):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    x = blocks(exponent, dtype, exponent + 500)
    if tall > 1:  # 128 rows a block: the borders in its first row, and other parts of the largest below them
        x = x[::9]
        parts = torch.linspace(1, 0.001, 128)[:, None]
        x = torch.cat([(row * parts).to(dtype) for row in x])
    want_c, want_s = ref.quantize(x.float().numpy(), tall)
    src = x.cuda()
    loose = torch.empty(x.shape[0], x.shape[1] + 5, dtype=dtype, device="cuda")[:, 3:-2]
    loose.copy_(src)
    for t in (src, loose):
        c, s = pulse.fp8_quantize(t, tall)
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)
        np.testing.assert_array_equal(c.view(torch.uint8).cpu().numpy(), want_c)
