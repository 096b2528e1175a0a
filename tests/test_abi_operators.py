"""CPU checks of the optimizer-step and logit-shaping entry points: bad
arguments are refused on the host before any CUDA call, and the binding refuses
wrong tensors."""
import ctypes

import pytest
import torch

import rl_post_trainer_gb300 as pulse
from rl_post_trainer_gb300 import _build

E = pulse.pulse
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pulse.lib()


def tensor(**kw):
    f = dict(n=8, master=16, grad=32, grad_dtype=0, m=64, v=128, m_exp=0, v_exp=0, m_out=0, v_out=0,
             weight_decay=0.0, lr_scale=1.0)
    f.update(kw)
    return (E.PulseAdamTensor * 1)(E.PulseAdamTensor(*f.values()))


def test_adam_plan_arguments(lib):
    h = P()
    create = lib.pulse_adam_plan_create
    assert create(None, 1, 32, ctypes.byref(h)) == E.PULSE_ERR_INVALID
    assert create(tensor(), 1, 32, None) == E.PULSE_ERR_INVALID
    for count in (0, -1, 16385):
        assert create(tensor(), count, 32, ctypes.byref(h)) == E.PULSE_ERR_INVALID
    for bits in (0, 16, 4):
        assert create(tensor(), 1, bits, ctypes.byref(h)) == E.PULSE_ERR_INVALID
    assert create(tensor(n=1 << 32), 1, 32, ctypes.byref(h)) == E.PULSE_ERR_RANGE
    inf, nan = float("inf"), float("nan")
    for bad in (dict(grad_dtype=2), dict(grad_dtype=-1), dict(weight_decay=-0.1), dict(weight_decay=inf),
                dict(weight_decay=nan), dict(lr_scale=-1.0), dict(lr_scale=nan), dict(master=18), dict(grad=33),
                dict(grad=33, grad_dtype=1), dict(grad=34), dict(m=65), dict(v=130), dict(m_out=2), dict(v_out=1)):
        assert create(tensor(**bad), 1, 32, ctypes.byref(h)) == E.PULSE_ERR_INVALID, bad
        assert not h.value


def test_adam_calls_without_a_plan(lib):
    hyper = E.PulseAdamHyper(1, 0, 1e-3, 0.9, 0.999, 1e-8)
    assert lib.pulse_adam_plan_destroy(None) == E.PULSE_OK
    assert lib.pulse_adam_plan_set_grads(None, (P * 1)(), P(0)) == E.PULSE_ERR_INVALID
    assert lib.pulse_grad_norm_multi(None, 1.0, P(8), P(8), P(0)) == E.PULSE_ERR_INVALID
    assert lib.pulse_adam_step_multi(None, ctypes.byref(hyper), P(0), P(0)) == E.PULSE_ERR_INVALID
    assert lib.pulse_adam_export_multi(None, P(0)) == E.PULSE_ERR_INVALID


def shaping(**kw):
    s = E.PulseLogitsShaping()
    s.vocab = 100
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


A, B, C = 1 << 20, 1 << 21, 1 << 22  # addresses that nothing reads


def test_shape_arguments(lib):
    def call(s=None, rows=4, src=A, stride=100, it=0, dst=B, ostride=100, ot=0):
        return lib.pulse_logits_shape(s or shaping(), rows, P(src), stride, it, P(dst), ostride, ot, P(0))
    assert lib.pulse_logits_shape(None, 4, P(A), 100, 0, P(B), 100, 0, P(0)) == E.PULSE_ERR_INVALID
    assert call(rows=0) == E.PULSE_OK
    assert call(rows=0, src=0, dst=0) == E.PULSE_OK
    for bad in (dict(src=0), dict(dst=0), dict(stride=99), dict(ostride=99), dict(stride=1 << 40), dict(it=2),
                dict(ot=2), dict(it=0, ot=1), dict(src=A + 2), dict(dst=B + 2), dict(src=A + 1, it=1, ot=1)):
        assert call(**bad) == E.PULSE_ERR_INVALID, bad
    for bad in (dict(vocab=0), dict(vocab=1 << 31), dict(tokens=8), dict(tokens=8, begin=8), dict(tokens=8, end=8),
                dict(tokens=8, begin=8, end=8, ntokens=1 << 62), dict(bias_tokens=8, bias_values=8),
                dict(bias_tokens=8, bias_begin=8), dict(bias_tokens=8, bias_begin=8, bias_values=8, nbias=1 << 31),
                dict(mask=8, mask_rows=1, mask_stride=3)):
        assert call(shaping(**bad)) == E.PULSE_ERR_INVALID, bad
    assert call(rows=1 << 40) == E.PULSE_ERR_RANGE
    assert lib.pulse_logits_shape(shaping(vocab=2 ** 31 - 1), 1 << 20, P(A), 1 << 31, 0, P(1 << 60), 1 << 31, 0,
                                  P(0)) == E.PULSE_ERR_RANGE


def test_shape_overlaps(lib):
    def call(src, dst, stride=100, ostride=100, it=0, ot=0, rows=4):
        return lib.pulse_logits_shape(shaping(), rows, P(src), stride, it, P(dst), ostride, ot, P(0))
    assert call(A, A + 4) == E.PULSE_ERR_INVALID                   # shifted by an element
    assert call(A, A, ostride=200) == E.PULSE_ERR_INVALID          # another pitch
    assert call(A, A, it=1, ot=0) == E.PULSE_ERR_INVALID           # another type
    assert call(A, A + 4 * 100 * 3) == E.PULSE_ERR_INVALID         # the last row
    assert call(A + 4 * 100 * 3, A) == E.PULSE_ERR_INVALID
    assert call(A, A + 4 * 99, stride=200, ostride=200) == E.PULSE_ERR_INVALID   # column ranges that meet
    assert call(A + 4 * 99, A, stride=200, ostride=200) == E.PULSE_ERR_INVALID
    assert call(A, A + 4 * 101, stride=200, ostride=200) == E.PULSE_ERR_INVALID  # wraps into the next row


def test_backward_arguments(lib):
    def call(s=None, rows=4, d=A, ds=100, ot=0, x=B, xs=100, it=0, o=C, os=100):
        return lib.pulse_logits_shape_backward(s or shaping(), rows, P(d), ds, ot, P(x), xs, it, P(o), os, P(0))
    assert call(rows=0) == E.PULSE_OK
    hist = dict(tokens=8, begin=8, end=8, ntokens=4, repetition=8)
    for bad in (dict(d=0), dict(o=0), dict(ds=99), dict(os=99), dict(it=0, ot=1), dict(d=A + 4, o=A), dict(it=3),
                dict(s=shaping(**hist), x=0), dict(s=shaping(**hist), xs=99), dict(s=shaping(**hist), x=C),
                dict(s=shaping(**hist), x=C + 4)):
        assert call(**bad) == E.PULSE_ERR_INVALID, bad
    assert call(rows=1 << 40) == E.PULSE_ERR_RANGE


def test_binding_refuses_cpu_tensors_and_bad_settings(lib):
    x = torch.zeros(8)
    with pytest.raises(ValueError):
        pulse.AdamPlan([])
    with pytest.raises(ValueError):
        pulse.AdamPlan([pulse.AdamTensorSlot(8, master=x)], state_bits=16)
    with pytest.raises(TypeError):
        pulse.AdamPlan([pulse.AdamTensorSlot(8, master=x)])
    with pytest.raises(TypeError):
        pulse.AdamTensorSlot(8, grad=torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        pulse.AdamPlan([pulse.AdamTensorSlot(0)])
    with pytest.raises(ValueError):
        pulse.LogitsPlan(-1, 10)
    with pytest.raises(ValueError):
        pulse.LogitsPlan(1, 0)
    with pytest.raises(ValueError):
        pulse.LogitsPlan(1, 10, tokens=x)
    with pytest.raises(ValueError):
        pulse.LogitsPlan(1, 10, bias_tokens=x)
    with pytest.raises(TypeError):
        pulse.LogitsPlan(1, 10, temperature=x)
    with pytest.raises(TypeError):
        pulse.LogitsPlan(1, 10, mask=torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(TypeError):
        pulse.LogitsPlan(1, 8).shape(x.reshape(1, 8))
    with pytest.raises(TypeError):
        pulse.LogitsPlan(1, 8).backward(x.reshape(1, 8))
    assert pulse.adam_blocks(0) == 0 and pulse.adam_blocks(1) == 1 and pulse.adam_blocks(257) == 2


def test_misaligned_settings_are_refused(lib):
    """Every list is read an element at a time: its pointer has to be aligned to that, used in the call or not."""
    full = dict(tokens=A, begin=A, split=A, end=A, ntokens=4, repetition=A, presence=A, frequency=A, temperature=A,
                bias_tokens=A, bias_values=A, bias_begin=A, nbias=4, mask=A, mask_rows=4, mask_stride=4, mask_row=A)
    for name, step in ((n, 4 if n in ("begin", "split", "end", "bias_begin") else 2) for n in full
                       if n not in ("ntokens", "nbias", "mask_rows", "mask_stride")):
        s = shaping(**{**full, name: A + step})
        assert lib.pulse_logits_shape(s, 4, P(B), 100, 0, P(C), 100, 0, P(0)) == E.PULSE_ERR_INVALID, name
        assert lib.pulse_logits_shape_backward(s, 4, P(B), 100, 0, P(2 * C), 100, 0, P(C), 100, P(0)) == E.PULSE_ERR_INVALID
        assert lib.pulse_logits_shape(s, 0, P(B), 100, 0, P(C), 100, 0, P(0)) == E.PULSE_ERR_INVALID, name
    assert lib.pulse_logits_shape(shaping(**full), 0, P(B), 100, 0, P(C), 100, 0, P(0)) == E.PULSE_OK


def test_sorts_arguments(lib):
    out = ctypes.c_int(7)
    assert lib.pulse_logits_sorts(None, 4, 0, ctypes.byref(out)) == E.PULSE_ERR_INVALID
    assert lib.pulse_logits_sorts(shaping(vocab=0), 4, 0, ctypes.byref(out)) == E.PULSE_ERR_INVALID
    assert lib.pulse_logits_sorts(shaping(), 4, 0, None) == E.PULSE_ERR_INVALID
    hist = dict(tokens=A, begin=A, end=A, ntokens=1 << 30)
    for s, rows, backward in ((shaping(), 4, 0), (shaping(**hist), 4, 0), (shaping(**hist, frequency=A), 4, 1),
                              (shaping(**hist, repetition=A), 0, 0)):
        out.value = 7
        assert lib.pulse_logits_sorts(s, rows, backward, ctypes.byref(out)) == E.PULSE_OK and out.value == 0
    assert lib.pulse_logits_sorts(shaping(**hist, repetition=A), 1 << 40, 0, ctypes.byref(out)) == E.PULSE_ERR_RANGE
