"""Shaping calls that sort their token lists first: every test asserts that its calls
do, and compares all rows with the unsorted way's bits and some with the float64
formulas."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import rl_post_trainer_gb300 as pulse
from test_gpu_logits import BF16, F32, NONE, PAIRS, WIDE, _cuda, plan_of, same, settings

pytestmark = pytest.mark.gpu


def subset(s, pick):
    """The settings of some rows alone."""
    out = dict(s)
    for k in ("begin", "split", "end", "repetition", "presence", "frequency", "temperature", "mask_row"):
        if s[k] is not None:
            out[k] = s[k][pick]
    if s["bias_tokens"] is not None:
        lists = [slice(int(s["bias_begin"][r]), int(s["bias_begin"][r + 1])) for r in pick]
        out["bias_tokens"] = np.concatenate([s["bias_tokens"][i] for i in lists])
        out["bias_values"] = np.concatenate([s["bias_values"][i] for i in lists])
        out["bias_begin"] = np.cumsum([0] + [i.stop - i.start for i in lists])
    return out


def unsorted(plan, x, d, y, dx):
    """The same calls as a graph has them, where nothing is sorted."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        plan.shape(x, out=y)
        plan.backward(d, logits=x, out=dx)
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()


def check_sorted(s, rows, vocab, tin, tout, pick, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 4).to(tin)
    d = torch.randn(rows, vocab, generator=gen, device="cuda").to(tout)
    plan = plan_of(s, rows, vocab)
    assert plan.sorts() and plan.sorts(backward=True)
    y, dx = plan.shape(x, out_dtype=tout), plan.backward(d, logits=x)
    assert pulse.get_error(torch.device("cuda", 0)) == 0
    few = subset(s, pick)
    want, size = ref.shape64(x[pick].double().cpu().numpy(), few)
    same(y[pick], want, size, tout)
    want = ref.shape64_backward(d[pick].double().cpu().numpy(), x[pick].double().cpu().numpy(), few)
    same(dx[pick], want, np.abs(want), tin)
    y2, dx2 = torch.zeros_like(y), torch.zeros_like(dx)
    unsorted(plan, x, d, y2, dx2)
    assert torch.equal(y, y2) and torch.equal(dx, dx2)


def text(g, n, vocab):
    """Words of a text: few of them often, most of them seldom."""
    return np.minimum(np.exp(g.random(n) * np.log(vocab)).astype(np.int64) - 1, vocab - 1).clip(0).astype(np.int32)


@pytest.mark.parametrize("tin,tout", PAIRS)
@pytest.mark.parametrize("rows,vocab", [(3000, 131075), (4096, 151936)])
@pytest.mark.parametrize("counts", [False, True])
def test_rows_of_one_sequence(tin, tout, rows, vocab, counts):
    """Training rows: row t has the tokens before it, all rows the same list."""
    _cuda()
    s = settings(rows, vocab, seed=51, bias=3 if counts else 0)
    if not counts:
        s.update({k: None for k in ("frequency", "presence", "bias_tokens", "bias_values", "bias_begin")})
    s["tokens"] = text(np.random.default_rng(1), rows, vocab)
    s["begin"], s["end"] = np.zeros(rows, np.int64), np.arange(rows)
    s["split"] = np.minimum(s["end"], 700)
    check_sorted(s, rows, vocab, tin, tout, [0, 1, 2, 699, 701, 2047, 2048, 2049, rows - 1])


@pytest.mark.parametrize("tin,tout", PAIRS)
@pytest.mark.parametrize("rows,vocab,history", [(2100, 16384, 4030), (400, 40000, 8500), (401, 40003, 8500),
                                                (80, 163840, 10600), (81, 160001, 10600)])
def test_few_slices_and_long_lists(tin, tout, rows, vocab, history):
    """2 to 20 slices a row, a list of its own for each row."""
    _cuda()
    g = np.random.default_rng(rows)
    s = settings(rows, vocab, seed=52, bias=20)
    s["begin"] = np.arange(rows) * history
    s["end"] = s["begin"] + history
    s["end"][3] = s["begin"][3]
    s["split"] = s["begin"] + (g.random(rows) * (s["end"] - s["begin"])).astype(np.int64)
    s["tokens"] = text(g, rows * history, vocab)
    check_sorted(s, rows, vocab, tin, tout, [0, 1, 3, 4, rows // 2, rows - 1])


@pytest.mark.parametrize("history", [1, 2, 2047, 2048, 2049, 4097, 9000])
def test_edges_of_blocks(history):
    """Histories that begin, split and end around the blocks of 2048 positions, and rows that share them."""
    _cuda()
    rows, vocab = 90, 150001
    g = np.random.default_rng(history)
    s = settings(rows, vocab, seed=53, bias=3)
    total = 2048 * 450 + 77
    s["tokens"] = text(g, total, vocab)
    s["begin"] = g.integers(0, total - history + 1, rows)
    s["begin"][:10] = [0, 1, 2047, 2048, 2049, 4095, 4096, 4097, total - history, total - 1]
    s["end"] = s["begin"] + history
    s["end"][9] = total
    s["end"][10] = s["begin"][10]
    s["split"] = s["begin"] + (np.arange(rows) * 37) % (s["end"] - s["begin"] + 1)
    check_sorted(s, rows, vocab, F32, F32, list(range(14)) + [rows - 1])


def test_bad_indices():
    """Tokens outside the vocabulary count as an error only inside a row's history."""
    dev = _cuda()
    rows, vocab = 400, 40000
    tokens = np.random.default_rng(3).integers(0, vocab, 3400000).astype(np.int32)
    tokens[[100, 2047, 2048]] = [-1, vocab, 2 ** 31 - 1]
    s = dict(NONE, tokens=tokens, repetition=np.full(rows, 2.0, np.float32))
    x = torch.randn(rows, vocab, device="cuda")
    pulse.get_error(dev)
    for begin, end, error in ((101, 2047, 0), (100, 200, 5), (2040, 2048, 5), (2048, 2049, 5), (2049, 3400000, 0), (0, 5000, 5)):
        s["begin"], s["end"] = np.full(rows, 0), np.full(rows, 0)
        s["begin"][333], s["end"][333] = begin, end
        plan = plan_of(s, rows, vocab)
        assert plan.sorts()
        y = plan.shape(x)
        assert pulse.get_error(dev) == error
        want, size = ref.shape64(x[333:334].cpu().numpy(), dict(s, begin=s["begin"][333:], end=s["end"][333:]))
        same(y[333:334], want, size, F32)
        assert torch.equal(y[:333], x[:333]) and torch.equal(y[334:], x[334:])


def test_what_the_kernel_in_front_writes():
    """Everything a sorted call reads is written right before it; the bits are those of calls with a wait after each."""
    _cuda()
    rows, vocab = 400, 40003
    s = settings(rows, vocab, seed=54, bias=20)
    s["begin"] = np.arange(rows) * 8500
    s["end"] = s["begin"] + 8500
    s["split"] = s["begin"] + 3000
    s["tokens"] = text(np.random.default_rng(4), rows * 8500, vocab)
    plan = plan_of(s, rows, vocab)
    assert plan.sorts() and plan.sorts(backward=True)
    first = {k: v.clone() for k, v in plan.tensors.items()}
    results = []
    for wait in (True, False):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        for k, v in plan.tensors.items():
            v.copy_(first[k])
        x = torch.randn(rows, vocab, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
        y, dx, seen = torch.zeros_like(x), torch.zeros_like(x), []
        t = plan.tensors
        for _ in range(12):
            for change in (lambda: x.mul_(0.9).add_(0.1), lambda: t["temperature"].add_(0.01), lambda: t["mask"].bitwise_not_(),
                           lambda: t["bias_values"].neg_(), lambda: t["end"].sub_(1), lambda: t["split"].add_(1),
                           lambda: t["repetition"].mul_(1.01), lambda: t["tokens"].add_(1).remainder_(vocab)):
                change()
                pause()
                plan.shape(x, out=y)
                pause()
                plan.backward(x, logits=x, out=dx)
                pause()
                seen += [y[::37, ::101].clone(), dx[::37, ::101].clone()]
        torch.cuda.synchronize()
        results.append(seen)
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_which_calls_sort():
    """The rule: many tokens and several waves of slices; and what the wide cases of test_gpu_logits.py reach."""
    _cuda()

    def plan(rows, vocab, tokens, **kw):
        z = torch.zeros(rows, dtype=torch.int64, device="cuda")
        f = {k: torch.ones(rows, device="cuda") for k in ("repetition", "frequency") if k not in kw}
        return pulse.LogitsPlan(rows, vocab, tokens=torch.zeros(tokens, dtype=torch.int32, device="cuda"), begin=z, end=z, **f)

    assert not plan(1, 151936, 32768).sorts()
    assert not plan(64, 128256, 64 * 256).sorts()
    big = plan(256, 128256, 256 * 8192)
    assert big.sorts() and big.sorts(256, backward=True) and not big.sorts(0) and not big.sorts(8)
    only = plan(256, 128256, 256 * 8192, repetition=None)
    assert only.sorts() and not only.sorts(backward=True)
    assert not pulse.LogitsPlan(256, 128256, temperature=torch.ones(256, device="cuda")).sorts()
    for history, seed in ((60000, 31), (60000, 34)):
        assert plan_of(settings(12, WIDE, history=history, seed=seed, bias=40), 12, WIDE).sorts()
    for total in (131072 + 4200, 140000):
        assert plan(12, WIDE, total).sorts()
