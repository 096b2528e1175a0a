"""Rows of logits as views: what counts as in place and what as an overlap."""
import numpy as np
import pytest
import torch

import rl_post_trainer_gb300 as pulse
from test_gpu_logits import BF16, F32, NONE, _cuda, plan_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_row_in_place_through_views_of_different_strides(dtype):
    """The stride of a single row means nothing: views that differ in it alone are the same row."""
    _cuda()
    vocab = 1003
    plan = plan_of(dict(NONE, temperature=np.full(1, 0.5, np.float32)), 1, vocab)
    both = torch.randn(2, 2 * vocab, device="cuda").to(dtype)
    want, other = plan.shape(both[:1, :vocab].clone()), both[:, vocab:].clone()
    wide, narrow = both[:1, :vocab], both[0, :vocab].unsqueeze(0)
    assert wide.stride() != narrow.stride() and wide.data_ptr() == narrow.data_ptr()
    assert plan.shape(wide, out=narrow) is narrow
    assert torch.equal(both[:1, :vocab], want) and torch.equal(both[:, vocab:], other)
    before = both[:1, :vocab].clone()
    plan.backward(narrow, out=wide)
    assert torch.equal(both[:1, :vocab], plan.backward(before)) and torch.equal(both[:, vocab:], other)
    with pytest.raises(pulse.PulseError):
        plan.shape(both[:1, :vocab], out=both[:1, 8:vocab + 8])
    plan.shape(both[:1, :vocab], out=both[:1, vocab:])
