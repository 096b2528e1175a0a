"""The FP8 product where a wait runs out: loaders that end early, on the device and with a short limit. The call returns, the
timeout is reported, nothing outside of the output is written, and the next call is right."""
import numpy as np
import pytest
import torch

import rl_post_trainer_gb300 as pulse
from test_gpu_fp8 import Rows, check_product, codes_of, on_gpu

pytestmark = pytest.mark.gpu

E = pulse.pulse
LIMIT = 20_000_000  # ns
# tokens, columns, outputs: 16, 32, 64 and 128 tokens a tile, sums split over clusters or not, tiles one after the other, pairs
SIZES = [(1, 300, 100), (5, 20000, 70), (3, 1500, 20011), (31, 3000, 300), (64, 4100, 1000), (128, 2003, 515), (400, 1280, 5003), (2049, 900, 1281)]


@pytest.mark.parametrize("m,k,n", SIZES)
def test_withheld_blocks(m, k, n):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    c, s = codes_of(m, k, 1, 1)
    w, sw = codes_of(n, k, 2, 128)
    x_c, w_c = on_gpu(c, (k + 31) // 16 * 16), on_gpu(w, (k + 47) // 16 * 16)
    x_s, w_s = torch.from_numpy(s).cuda(), torch.from_numpy(sw).cuda()
    out = Rows(m, n, torch.float32, n + 3, 1)
    blocks = (k + 127) // 128
    assert pulse.get_error() == E.PULSE_OK
    for loaders in (1, 2, 3, 4, 8, 15):
        for block in sorted({0, 1, 2, 6, blocks // 2}):
            E.debug_fp8_linear_withheld(x_c, x_s, w_c, w_s, out.t, loaders, block, LIMIT)
            torch.cuda.synchronize()
            error = pulse.get_error()
            out.check()
            if loaders & 3 and block == 0:  # every CTA has a first block
                assert error == E.PULSE_ERR_TIMEOUT
            assert error in (E.PULSE_OK, E.PULSE_ERR_TIMEOUT)
            if error == E.PULSE_OK:  # no CTA has such a block, or such loaders
                check_product(c, s, w, sw, out.t, torch.float32)
        pulse.fp8_linear(x_c, x_s, w_c, w_s, out.t)
        assert pulse.get_error() == E.PULSE_OK
        check_product(c, s, w, sw, out.t, torch.float32)
        out.check()
    E.debug_fp8_linear_withheld(x_c, x_s, w_c, w_s, out.t, 15, 1 << 31, 1_000_000_000)  # no such block
    assert pulse.get_error() == E.PULSE_OK
    check_product(c, s, w, sw, out.t, torch.float32)


def test_another_stream_goes_on():
    """A product that gives up on one stream leaves the ones on another as they are."""
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    c, s = codes_of(300, 1000, 1, 1)
    w, sw = codes_of(3000, 1000, 2, 128)
    x_c, w_c = on_gpu(c), on_gpu(w)
    x_s, w_s = torch.from_numpy(s).cuda(), torch.from_numpy(sw).cuda()
    want = pulse.fp8_linear(x_c, x_s, w_c, w_s)
    bad = torch.empty(300, 3000, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            E.debug_fp8_linear_withheld(x_c, x_s, w_c, w_s, bad, 2, 3, LIMIT)
        with torch.cuda.stream(streams[1]):
            got += [pulse.fp8_linear(x_c, x_s, w_c, w_s) for _ in range(5)]
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        assert pulse.get_error() == E.PULSE_ERR_TIMEOUT
    with torch.cuda.stream(streams[1]):
        assert pulse.get_error() == E.PULSE_OK
    assert all(torch.equal(want, g) for g in got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,k,n", [(129, 1000, 10001), (400, 2003, 5003), (2049, 128, 1281), (513, 5000, 4000), (3000, 300, 20011)])
def test_many_tokens_without_pairs(m, k, n, dtype):
    """What a build whose pair kernel has too few registers does instead."""
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    c, s = codes_of(m, k, 1, 1, wild=m % 2 == 1)
    w, sw = codes_of(n, k, 2, 128)
    for pitch, shift in ((n, 0), (n + 3, 1)):
        out = Rows(m, n, dtype, pitch, shift)
        x_c, w_c, x_s, w_s = on_gpu(c, (k + 31) // 16 * 16), on_gpu(w), torch.from_numpy(s).cuda(), torch.from_numpy(sw).cuda()
        E.debug_fp8_linear_withheld(x_c, x_s, w_c, w_s, out.t, 16, 0, 1_000_000_000)
        torch.cuda.synchronize()
        check_product(c, s, w, sw, out.t, dtype)
        out.check()
    assert pulse.get_error() == E.PULSE_OK
