"""RMS norm of rows whose squares pass FP32's range at either end, alone and beside ordinary rows."""
import numpy as np
import pytest
import torch

import rl_post_trainer_gb300 as pulse
from test_gpu_fp8 import check_norm, host, values

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def rows_of(cols, dtype, seed):
    """Ordinary rows, and rows from the smallest numbers of the type to the largest: every sum of squares that FP32 does not hold."""
    x = values(9, cols, dtype, seed, special=False).float()
    x = x / x.abs().amax(1, keepdim=True).clamp(min=1e-30)
    size = [1.0, 2.0 ** -60, 2.0 ** -64, 2.0 ** -75, 2.0 ** -100, 2.0 ** -130, 2.0 ** 63, 2.0 ** 100, 2.0 ** 127]
    return (x.double() * torch.tensor(size, dtype=torch.float64)[:, None]).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [1, 128, 1003, 1536, 8192, 8200, 12000, 16385, 20000])
def test_small_and_large_rows(cols, dtype):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    x = rows_of(cols, dtype, cols)
    g = 1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(1))
    for eps in (0.0, 1e-44, 1e-38, 1e-30, 1e-12):
        check_norm(x, None, g, float(np.float32(eps)), pulse.rmsnorm_fp8(x.cuda(), g.cuda(), eps), dtype)
    # halves that add up to the row, in place and off 16 bytes
    half = (x.double() / 2).to(dtype)
    wide = torch.empty(9, cols + 3, dtype=dtype, device="cuda")[:, 1:-2]
    wide.copy_(half)
    res = half.cuda()
    got = pulse.rmsnorm_fp8(wide, g.cuda().to(BF16), 0.0, residual=res, sum_out=res)
    check_norm(half, half, g.to(BF16), 0.0, got, dtype)


def test_zeros_and_not_finite_without_eps():
    """A row of zeros has no norm where eps is 0; an infinity or a NaN leaves the other rows as they are."""
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    x = rows_of(700, F32, 3)
    clean = pulse.rmsnorm_fp8(x.cuda(), None, 0.0)
    bad = x.clone()
    bad[1], bad[3, 300], bad[6, 5] = 0.0, float("nan"), float("inf")
    c, s, _ = pulse.rmsnorm_fp8(bad.cuda(), None, 0.0)
    c, s = host(c.contiguous()), host(s)
    assert np.isnan(s[1]).all() and (c[1] == 0x7F).all() and np.isnan(s[3]).all()
    assert np.isnan(s[6, 0]) and (c[6, :128] == 0x7F).all()
    keep = [0, 2, 4, 5, 7, 8]
    np.testing.assert_array_equal(c[keep], host(clean[0].contiguous())[keep])
    np.testing.assert_array_equal(s[keep], host(clean[1])[keep])
