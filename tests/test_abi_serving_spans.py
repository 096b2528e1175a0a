"""Matrices whose rows lie so far apart that no address range holds them are refused on the host, before any CUDA call."""
import ctypes

import pytest

import rl_post_trainer_gb300 as pulse
from rl_post_trainer_gb300 import _build

P = ctypes.c_void_p
A, B, C, D, F, G = (k << 28 for k in range(1, 7))  # addresses that nothing reads
INVALID = pulse.pulse.PULSE_ERR_INVALID
# (rows - 1) * stride * 4 passes 2^64 for some, and comes out small or behind the matrix's own beginning
FAR = [(1 << 30, 1 << 34), (1 << 25, 1 << 39), ((1 << 25) + 1, 1 << 39), ((1 << 26) - 1, (1 << 40) - 16), ((1 << 24) + 1, 1 << 38), ((1 << 17) + 1, 1 << 39)]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pulse.lib()


@pytest.mark.parametrize("rows,stride", FAR)
def test_far_rows_are_refused(lib, rows, stride):
    for x, c, s in ((stride, 16, 1), (16, stride, 1), (16, 16, stride)):
        assert lib.pulse_fp8_quantize(P(A), rows, 16, x, 0, 1, P(B), c, P(C), s, P(0)) == INVALID
    for st in ((stride, 16, 16), (16, stride, 16), (16, 16, stride)):
        assert lib.pulse_rmsnorm_fp8(P(A), rows, 16, st[0], 1, P(B), st[1], P(C), st[2], P(D), 0, 0.0, P(F), 16, P(G), 1, P(0)) == INVALID
    for m, n, xs, sxs, ws, sws, os in ((rows, 16, stride, 1, 16, 1, 16), (rows, 16, 16, stride, 16, 1, 16), (1, rows, 16, 1, stride, 1, rows),
                                       (rows, 16, 16, 1, 16, 1, stride), (1, rows << 1, 16, 1, 16, stride << 1, rows << 1)):
        if n < 1 << 31:
            assert lib.pulse_fp8_linear(P(A), m, xs, P(B), sxs, P(C), n, ws, P(D), sws, 16, P(F), os, 0, P(0)) == INVALID
    if rows < 1 << 26:
        assert lib.pulse_sample(ctypes.byref(pulse.pulse.PulseSampling(16)), rows, P(A), stride, 0, P(0x7 << 40), P(0x7 << 41), P(0), P(0)) == INVALID
