"""LogitsPlan.shape under autograd: the gradient of the shaped logits is that of
LogitsPlan.backward, and what would make it wrong is refused."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import rl_post_trainer_gb300 as pulse
from test_gpu_logits import BF16, F32, NONE, PAIRS, _cuda, plan_of, same, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tin,tout", PAIRS)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 33), (5, 5003), (40, 2049)])
@pytest.mark.parametrize("without", [(), ("repetition",), ("tokens", "begin", "split", "end")])
def test_gradient_through_shape(tin, tout, rows, vocab, without):
    _cuda()
    s = settings(rows, vocab, seed=41, **{k: None for k in without})
    plan = plan_of(s, rows, vocab)
    x = (torch.randn(rows, vocab, device="cuda") * 4).to(tin).requires_grad_()
    y = plan.shape(x, out_dtype=tout)
    assert y.requires_grad and y.dtype == tout
    with torch.no_grad():
        bare = plan.shape(x, out_dtype=tout)
    assert not bare.requires_grad and torch.equal(y, bare) and torch.equal(plan.shape(x.detach(), out_dtype=tout), bare)
    d = torch.randn(rows, vocab, device="cuda").to(tout)
    y.backward(d)
    assert x.grad.dtype == tin
    want = ref.shape64_backward(d.double().cpu().numpy(), x.detach().double().cpu().numpy(), s)
    same(x.grad, want, np.abs(want), tin)


def test_gradient_of_a_loss():
    """Through a log-softmax, from non-leaf logits, and with a broadcast incoming gradient."""
    _cuda()
    rows, vocab = 7, 1003
    s = settings(rows, vocab, seed=42)
    s["mask_row"] = np.full(rows, -1, np.int32)
    plan = plan_of(s, rows, vocab)
    h = torch.randn(rows, 16, device="cuda", requires_grad=True)
    w = torch.randn(vocab, 16, device="cuda")
    pick = torch.randint(0, vocab, (rows, 1), device="cuda")
    torch.log_softmax(plan.shape(h @ w.t()), -1).gather(1, pick).sum().backward()
    x = (h.detach() @ w.t()).requires_grad_()
    shaped = plan.shape(x.detach())
    d = -torch.softmax(shaped, -1)
    d.scatter_add_(1, pick, torch.ones_like(d[:, :1]))
    dx = plan.backward(d, logits=x.detach())
    # FP32 sums over the vocabulary, about 1000 terms in any order, of products with |w| up to about 5
    assert torch.allclose(h.grad, dx @ w, rtol=1e-4, atol=1e-4)
    plan.shape(x).sum().backward()  # its incoming gradient has strides of 0
    assert torch.equal(x.grad, plan.backward(torch.ones_like(x), logits=x.detach()))


def test_settings_changed_before_the_backward_pass():
    """A wrong gradient is refused; settings that the gradient does not read may move."""
    _cuda()
    rows, vocab = 4, 500
    s = settings(rows, vocab, seed=43)
    x = torch.randn(rows, vocab, device="cuda", requires_grad=True)
    d = torch.ones(rows, vocab, device="cuda")
    for name in ("tokens", "end", "repetition", "temperature", "mask", "mask_row", "frequency", "bias_values"):
        plan = plan_of(s, rows, vocab)
        y = plan.shape(x)
        plan.tensors[name].add_(0)
        if name in ("frequency", "bias_values"):
            y.backward(d)
        else:
            with pytest.raises(RuntimeError, match="inplace"):
                y.backward(d)
    plan = plan_of(dict(s, repetition=None), rows, vocab)  # the history is counted only
    y = plan.shape(x)
    plan.tensors["tokens"].add_(0), plan.tensors["end"].add_(0)
    y.backward(d)
    plan = plan_of(s, rows, vocab)
    z = x * 1
    y = plan.shape(z)
    z.mul_(2)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward(d)


def test_given_buffers_carry_no_gradient():
    _cuda()
    plan = plan_of(dict(NONE, temperature=np.full(2, 0.5, np.float32)), 2, 64)
    x = torch.randn(2, 64, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        plan.shape(x, out=torch.empty(2, 64, device="cuda"))
    with pytest.raises(ValueError):
        plan.shape(x * 1, out=torch.empty(2, 64, device="cuda"))
    with torch.no_grad():
        out = torch.empty(2, 64, device="cuda")
        assert plan.shape(x, out=out) is out and torch.equal(out, x * 2)
    with pytest.raises(TypeError):
        plan.shape(x, out_dtype=BF16)
    with pytest.raises(ValueError):
        plan.shape(torch.zeros(2, 65, device="cuda", requires_grad=True))
    assert plan.shape(torch.zeros(0, 64, device="cuda", requires_grad=True)).shape == (0, 64)
    # no history or penalty: the gradient needs no logits and keeps none
    y = plan.shape(x.to(BF16), out_dtype=F32)
    y.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))


@pytest.mark.parametrize("call", ["shape", "backward"])
def test_in_place_calls_are_seen_by_autograd(call):
    """A tensor that a backward pass needs and that a call changed in place makes that pass fail."""
    _cuda()
    plan = plan_of(dict(NONE, temperature=np.full(2, 0.5, np.float32)), 2, 64)
    run = plan.shape if call == "shape" else plan.backward
    w = torch.ones(2, 64, device="cuda", requires_grad=True)
    for in_place in (False, True):
        x = torch.randn(2, 64, device="cuda")
        y = (w * x).sum()
        run(x, out=x if in_place else torch.empty_like(x))
        if in_place:
            with pytest.raises(RuntimeError, match="inplace"):
                y.backward()
        else:
            y.backward()
    with torch.inference_mode():
        x = torch.randn(2, 64, device="cuda")
        want = x * 2
        assert torch.equal(run(x, out=x), want)
