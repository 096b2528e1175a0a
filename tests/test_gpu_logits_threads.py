"""Shaping calls of several host threads on one stream: the library's sorted
histories belong to the stream, and every call has to read its own."""
import threading

import numpy as np
import pytest
import torch

import rl_post_trainer_gb300 as pulse

pytestmark = pytest.mark.gpu

VOCAB = 1100000  # many slices a row, so that a few rows with long histories are sorted


def _plan(rows, history, seed):
    g = np.random.default_rng(seed)
    dev = torch.device("cuda", 0)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    begin = np.arange(rows) * history
    return pulse.LogitsPlan(rows, VOCAB, device=dev, tokens=up(g.integers(0, VOCAB, rows * history).astype(np.int32)),
                            begin=up(begin), split=up(begin + history // 3), end=up(begin + history),
                            repetition=up((1.1 + g.random(rows)).astype(np.float32)),
                            frequency=up(g.random(rows).astype(np.float32)))


@pytest.mark.parametrize("stream", ["default", "side"])
def test_threads_on_one_stream(stream):
    """Two threads with different plans of sorting size, the second's ever larger, so that the workspace grows meanwhile."""
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    rows = 12
    small, large = [_plan(rows, 12000, 1)], [_plan(rows, 12000 * k, k) for k in (2, 3, 4, 5, 6)]
    x = torch.randn(rows, VOCAB, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    # alone, each on a stream of its own, so that the shared stream's workspace starts empty
    want = {}
    for p in small + large:
        with torch.cuda.stream(torch.cuda.Stream()):
            want[p] = (p.shape(x), p.backward(x, logits=x))
            torch.cuda.synchronize()
    shared = torch.cuda.current_stream() if stream == "default" else torch.cuda.Stream()
    wrong, failed = [], []

    def work(plans, rounds):
        try:
            out, dx = torch.empty_like(x), torch.empty_like(x)
            with torch.cuda.stream(shared):
                for p in plans:
                    for _ in range(rounds):
                        p.shape(x, out=out)
                        p.backward(x, logits=x, out=dx)
                        if not (torch.equal(out, want[p][0]) and torch.equal(dx, want[p][1])):
                            wrong.append(p)
        except Exception as e:  # a thread's exception would go unseen
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in ((small, 50), (large, 10))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert not wrong
    assert pulse.get_error(torch.device("cuda", 0)) == 0


def test_threads_on_their_default_streams():
    """cudaStreamPerThread: one handle, a stream of its own in every thread."""
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    rows, per_thread = 12, 2
    plans = [_plan(rows, 12000 * k, k) for k in (1, 2, 3)]
    x = torch.randn(rows, VOCAB, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    want = [p.shape(x) for p in plans]
    outs = [[torch.zeros_like(x) for _ in range(10)] for _ in plans]
    torch.cuda.synchronize()
    status = []

    def work(p, many):
        torch.cuda.set_device(0)
        for out in many:
            status.append(pulse.lib().pulse_logits_shape(p._ref, rows, x.data_ptr(), VOCAB, 0, out.data_ptr(), VOCAB, 0, per_thread))

    threads = [threading.Thread(target=work, args=a) for a in zip(plans, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [0] * 30
    assert all(torch.equal(out, y) for many, y in zip(outs, want) for out in many)
