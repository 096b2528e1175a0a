"""The FP8 product with scales whose own product leaves FP32's range: multiplied first, as documented."""
import numpy as np
import pytest
import torch

import rl_post_trainer_gb300 as pulse
import serving_ref as ref
from test_gpu_fp8 import host, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", [(3, 300), (40, 300), (300, 300), (310, 4400), (650, 5400)])
def test_scales_are_multiplied_first(m, n):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    g = np.random.default_rng(m)
    k = 512
    x, w = g.integers(1, 9, (m, k)), g.integers(1, 9, (n, k))  # sums of a block are whole numbers
    sx, sw = np.ones((m, 4), np.float32), np.ones((ref.blocks_of(n), 4), np.float32)
    sx[:, 1:], sx[1, 0], sx[2, 0], sx[0, 0] = 0, 2.0 ** 100, 2.0 ** -100, 3 * 2.0 ** -75
    sw[0, 0], sw[1, 0], sw[2, 0] = 2.0 ** 100, 2.0 ** -100, 2.0 ** -74
    out = pulse.fp8_linear(on_gpu(ref.e4m3_codes(x)), torch.from_numpy(sx).cuda(), on_gpu(ref.e4m3_codes(w)), torch.from_numpy(sw).cuda(),
                           out_dtype=torch.float32)
    with np.errstate(all="ignore"):
        first = sx[:, :1] * np.repeat(sw[:, 0], 128)[None, :n]  # FP32: infinite, 0, or two bits of 3 * 2^-149
        want = first * (x[:, :128] @ w[:, :128].T).astype(np.float32)
    assert np.isinf(want).any() and (want == 0).any()
    np.testing.assert_array_equal(host(out), want)
    assert pulse.get_error() == 0
