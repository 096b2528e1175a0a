"""Arguments that the test hook of the FP8 product refuses before any CUDA call."""
import ctypes

import rl_post_trainer_gb300 as pulse
from rl_post_trainer_gb300 import _build

P = ctypes.c_void_p
A, B, C, D, F = (k << 28 for k in range(1, 6))  # addresses that nothing reads


def test_withheld_arguments():
    _build.build()

    def call(loaders=1, limit=1000, m=4, xs=320):
        return pulse.lib().pulse_debug_fp8_linear_withheld(P(A), m, xs, P(B), 3, P(C), 200, 320, P(D), 3, 300, P(F), 200, 0, loaders, 0, limit, P(0))
    for bad in (dict(loaders=0), dict(loaders=32), dict(limit=1_000_000_001), dict(xs=312)):
        assert call(**bad) == pulse.pulse.PULSE_ERR_INVALID, bad
    assert call(m=0) == pulse.pulse.PULSE_OK
