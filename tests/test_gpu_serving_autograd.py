"""Buffers that the FP8 path and the sampling overwrite are known to autograd, and what carries a tangent is refused."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import rl_post_trainer_gb300 as pulse

pytestmark = pytest.mark.gpu

F32, F8 = torch.float32, torch.float8_e4m3fn


def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    return torch.device("cuda", 0)


def calls():
    """(name, call that overwrites its argument, the argument) for every output of every operator."""
    dev = _cuda()
    x, res = torch.randn(4, 256, device=dev), torch.randn(4, 256, device=dev)
    codes, scales = pulse.fp8_quantize(x)
    plan = pulse.SamplePlan(4, 256)
    u = torch.rand(4, device=dev)

    def c():
        return torch.zeros(4, 256, dtype=F8, device=dev)

    def s():
        return torch.zeros(4, 2, device=dev)
    wide = pulse.fp8_quantize(x, pulse.FP8_BLOCK)
    return [("quantize codes", lambda t: pulse.fp8_quantize(x, 1, t), c()),
            ("quantize scales", lambda t: pulse.fp8_quantize(x, 1, None, t), s()),
            ("norm codes", lambda t: pulse.rmsnorm_fp8(x, None, codes_out=t), c()),
            ("norm scales", lambda t: pulse.rmsnorm_fp8(x, None, scales_out=t), s()),
            ("norm sum", lambda t: pulse.rmsnorm_fp8(x, None, residual=res, sum_out=t), torch.zeros(4, 256, device=dev)),
            ("norm sum in place", lambda t: pulse.rmsnorm_fp8(t, None, residual=res, sum_out=t), torch.zeros(4, 256, device=dev)),
            ("linear", lambda t: pulse.fp8_linear(codes, scales, *wide, out=t), torch.zeros(4, 4, device=dev)),
            ("tokens", lambda t: plan.sample(x, u, t), torch.zeros(4, dtype=torch.int32, device=dev)),
            ("logprobs", lambda t: plan.sample(x, u, None, t), torch.zeros(4, device=dev))]


def test_versions():
    for name, call, t in calls():
        before = t._version
        call(t)
        assert t._version > before, name
        with torch.inference_mode():
            call(torch.zeros_like(t))  # has no version


def test_backward_of_an_overwritten_buffer_fails():
    for name, call, t in calls():
        if t.dtype != F32:
            continue
        w = torch.ones(t.shape, device="cuda", requires_grad=True)
        loss = (w * t).sum()  # saves t
        call(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    table = torch.zeros(4, 300, device="cuda", requires_grad=True)
    tokens = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss = table.index_select(1, tokens).sum()  # saves the tokens
    pulse.SamplePlan(4, 256).sample(torch.randn(4, 256, device="cuda"), torch.rand(4, device="cuda"), tokens)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_that_require_a_gradient_are_refused():
    for name, call, t in calls():
        if t.dtype != F32:
            continue
        t.requires_grad_()
        with pytest.raises(ValueError):
            call(t)
        with torch.no_grad():
            call(t)


def test_tangents_are_refused():
    dev = _cuda()
    x, g = torch.randn(4, 256, device=dev), torch.ones(256, device=dev)
    codes, scales = pulse.fp8_quantize(x)
    wide, wide_scales = pulse.fp8_quantize(x, pulse.FP8_BLOCK)
    u = torch.rand(4, device=dev)
    with fwd.dual_level():
        def dual(t):
            return fwd.make_dual(t, torch.ones_like(t))
        for call in (lambda: pulse.fp8_quantize(dual(x)), lambda: pulse.rmsnorm_fp8(dual(x), g), lambda: pulse.rmsnorm_fp8(x, dual(g)),
                     lambda: pulse.rmsnorm_fp8(x, g, residual=dual(x)), lambda: pulse.fp8_linear(codes, dual(scales), wide, wide_scales),
                     lambda: pulse.fp8_linear(codes, scales, wide, dual(wide_scales)),
                     lambda: pulse.SamplePlan(4, 256).sample(x, u, logprobs_out=dual(u))):
            with pytest.raises(ValueError, match="tangent"):
                call()
        pulse.fp8_quantize(x), pulse.rmsnorm_fp8(x, g)  # without one they run
        tokens, logprobs = pulse.SamplePlan(4, 256).sample(dual(x), u)  # as logits that require a gradient: taken, and none given
        assert fwd.unpack_dual(logprobs).tangent is None


def test_function_transforms_are_refused():
    """torch.func hands out tensors without memory of their own: an error, not a gradient of zero."""
    x = torch.randn(4, 256, device=_cuda())
    for call in (lambda t: pulse.fp8_quantize(t)[1].sum(), lambda t: pulse.rmsnorm_fp8(t, None)[1].sum()):
        with pytest.raises((RuntimeError, ValueError)):
            torch.func.grad(call)(x)
        with pytest.raises((RuntimeError, ValueError)):
            torch.func.jvp(call, (x,), (torch.ones_like(x),))
