"""Logit shaping and its gradient on the GPU against the float64 formulas:
ragged and empty histories, odd vocabularies, strided and misaligned rows, masks
that leave a row empty, non-finite values in masked places, bad indices."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import rl_post_trainer_gb300 as pulse
from pulse_testutil import Guarded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PAIRS = [(F32, F32), (BF16, BF16), (BF16, F32)]
# FP32: at most 8 roundings of the terms' size (penalty, count product, two differences, bias, reciprocal, product,
# the temperature's own). A BF16 output is the rounding of a value inside that interval: rounding keeps order, so it lies
# between the roundings of the interval's ends
TOL32 = 8 * 2.0 ** -24


def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    return torch.device("cuda", 0)


def settings(rows, vocab, history=50, seed=0, empty=True, bias=5, masks=3, **without):
    """Random settings of every kind; `without=...=None` leaves one out."""
    g = np.random.default_rng(seed)
    lens = g.integers(0 if empty else 1, history + 1, rows)
    end = np.cumsum(lens)
    begin = end - lens
    split = begin + (lens * g.random(rows)).astype(np.int64)
    tokens = np.minimum(np.exp(g.random(max(1, int(lens.sum()))) * np.log(vocab + 1)).astype(np.int64) - 1, vocab - 1)
    words = (vocab + 31) // 32
    s = dict(tokens=np.maximum(tokens, 0).astype(np.int32), begin=begin.astype(np.int64), split=split.astype(np.int64),
             end=end.astype(np.int64), repetition=(0.7 + g.random(rows)).astype(np.float32),
             presence=g.normal(0, 1, rows).astype(np.float32), frequency=g.normal(0, .5, rows).astype(np.float32),
             temperature=(0.3 + 2 * g.random(rows)).astype(np.float32),
             bias_tokens=g.integers(0, vocab, rows * bias).astype(np.int32),
             bias_values=g.normal(0, 5, rows * bias).astype(np.float32),
             bias_begin=(np.arange(rows + 1) * bias).astype(np.int64),
             mask=g.integers(-2 ** 31, 2 ** 31, (masks, words)).astype(np.int32),
             mask_row=g.integers(-1, masks, rows).astype(np.int32))
    if rows > 2:
        s["temperature"][1] = 0.0
    s["mask"][0] = 0
    s.update(without)
    return s


NONE = dict(tokens=None, begin=None, split=None, end=None, repetition=None, presence=None, frequency=None,
            temperature=None, bias_tokens=None, bias_values=None, bias_begin=None, mask=None, mask_row=None)


def plan_of(s, rows, vocab):
    dev = torch.device("cuda", 0)
    return pulse.LogitsPlan(rows, vocab, device=dev, **{
        k: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(dev) for k, v in s.items()})


class Rows:
    """rows x vocab of `dtype` inside a guarded buffer: row pitch and first element as asked."""

    def __init__(self, rows, vocab, dtype, pitch=None, shift=0, init=None):
        self.pitch = pitch or vocab
        self.box = Guarded(rows * self.pitch + shift, dtype)
        self.t = torch.as_strided(self.box.t, (rows, vocab), (self.pitch, 1), self.box.t.storage_offset() + shift)
        if init is not None:
            self.t.copy_(init)
        self.before = self.box.t.clone()

    def check(self):
        """Nothing between the rows was written."""
        self.box.check()
        now = self.box.t.clone()
        keep = torch.as_strided(now, self.t.shape, self.t.stride(), self.t.storage_offset() - self.box.t.storage_offset())
        old = torch.as_strided(self.before, self.t.shape, self.t.stride(), self.t.storage_offset() - self.box.t.storage_offset())
        keep.copy_(old)
        assert torch.equal(now.view(torch.uint8), self.before.view(torch.uint8))


def same(got, want, size, dtype):
    got = got.double().cpu().numpy()
    ok = np.isfinite(want)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(got[~ok & ~np.isnan(want)], want[~ok & ~np.isnan(want)])
    got, want, tol = got[ok], want[ok], size[ok] * TOL32 + 1e-44
    lo, hi = want - tol, want + tol
    if dtype == BF16:  # the ends go outwards to FP32 first, so that they are rounded to BF16 once
        lo, hi = (torch.from_numpy(np.nextafter(e.astype(np.float32), np.float32(far))).to(BF16).double().numpy()
                  for e, far in ((lo, -np.inf), (hi, np.inf)))
    assert np.all((lo <= got) & (got <= hi)), np.max(np.abs(got - want) / tol)


def check(s, rows, vocab, tin, tout, x=None, pitch=(None, None, None), shift=(0, 0, 0), seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if x is None:
        x = torch.randn(rows, vocab, generator=gen, device="cuda") * 4
    src = Rows(rows, vocab, tin, pitch[0], shift[0], x.to(tin))
    dst = Rows(rows, vocab, tout, pitch[1], shift[1])
    plan = plan_of(s, rows, vocab)
    got = plan.shape(src.t, out=dst.t)
    assert got is dst.t
    want, size = ref.shape64(src.t.double().cpu().numpy(), s)
    same(got, want, size, tout)
    dst.check(), src.check()
    assert torch.equal(src.box.t.view(torch.uint8), src.before.view(torch.uint8))
    # backward
    d = Rows(rows, vocab, tout, pitch[1], shift[1], torch.randn(rows, vocab, generator=gen, device="cuda").to(tout))
    dx = Rows(rows, vocab, tin, pitch[2], shift[2])
    plan.backward(d.t, logits=src.t, out=dx.t)
    want = ref.shape64_backward(d.t.double().cpu().numpy(), src.t.double().cpu().numpy(), s)
    same(dx.t, want, np.abs(want), tin)
    dx.check(), d.check(), src.check()
    assert pulse.get_error(torch.device("cuda", 0)) == 0


@pytest.mark.parametrize("tin,tout", PAIRS)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (1, 31), (3, 32), (2, 33), (5, 1000), (4, 4096), (3, 4097), (2, 32003),
                                        (7, 8191), (1, 151936), (40, 2049)])
def test_everything_at_once(tin, tout, rows, vocab):
    _cuda()
    check(settings(rows, vocab, seed=rows + vocab), rows, vocab, tin, tout)


@pytest.mark.parametrize("tin,tout", PAIRS)
@pytest.mark.parametrize("keys", [(), ("tokens", "repetition"), ("tokens", "presence"), ("tokens", "frequency"),
                                  ("tokens", "frequency", "presence"), ("bias",), ("mask",), ("temperature",), ("tokens",),
                                  ("mask", "temperature", "bias"), ("repetition",)])
def test_each_setting_alone(tin, tout, keys):
    _cuda()
    full = settings(6, 5003, seed=3)
    names = {"tokens": ("tokens", "begin", "split", "end"), "bias": ("bias_tokens", "bias_values", "bias_begin"),
             "mask": ("mask", "mask_row")}
    s = dict(NONE)
    for k in keys:
        for n in names.get(k, (k,)):
            s[n] = full[n]
    check(s, 6, 5003, tin, tout)


@pytest.mark.parametrize("tin,tout", PAIRS)
@pytest.mark.parametrize("pitch,shift", [((2100, 2100, 2100), (0, 0, 0)), ((2055, 2060, 2049), (1, 3, 2)),
                                         ((2056, 2064, 2056), (8, 8, 8)), ((2056, 2056, 2056), (4, 4, 4)),
                                         ((2053, 2053, 2053), (5, 5, 5)), ((4100, 2049, 3000), (1, 0, 7))])
def test_strides_and_alignment(tin, tout, pitch, shift):
    _cuda()
    check(settings(9, 2049, seed=4), 9, 2049, tin, tout, pitch=pitch, shift=shift)


@pytest.mark.parametrize("history", [0, 1, 2, 255, 256, 257, 5000, 40000])
def test_history_lengths(history):
    _cuda()
    s = settings(3, 3001, history=max(1, history), seed=5, empty=history == 0)
    n = 3 * history
    g = np.random.default_rng(history)
    s["tokens"] = g.integers(0, 3001, max(1, n)).astype(np.int32)
    s["begin"] = np.arange(3) * history
    s["end"] = s["begin"] + history
    s["split"] = s["begin"] + np.array([0, history // 2, history])
    check(s, 3, 3001, BF16, F32)


def test_one_token_generated_very_often():
    _cuda()
    s = dict(NONE, tokens=np.full(100000, 7, np.int32), begin=np.array([0]), end=np.array([100000]),
             frequency=np.array([1e-3], np.float32), presence=np.array([2.0], np.float32))
    check(s, 1, 50, F32, F32)


def test_prefixes_of_one_sequence():
    """Training rows: row t has the tokens before it, all in one buffer."""
    _cuda()
    rows = 300
    s = settings(rows, 777, seed=6)
    s["tokens"] = np.random.default_rng(1).integers(0, 777, rows).astype(np.int32)
    s["begin"] = np.zeros(rows, np.int64)
    s["end"] = np.arange(rows)
    s["split"] = np.minimum(s["end"], 40)
    check(s, rows, 777, F32, F32)


def test_split_left_out_counts_all_as_generated():
    _cuda()
    s = settings(4, 500, seed=7)
    s["split"] = None
    check(s, 4, 500, F32, F32)


def test_token_biased_twice_takes_the_last_entry():
    _cuda()
    n = 3000
    g = np.random.default_rng(2)
    s = dict(NONE, bias_tokens=g.integers(0, 9, n).astype(np.int32), bias_values=g.normal(0, 1, n).astype(np.float32),
             bias_begin=np.array([0, n // 2, n]))
    for _ in range(3):
        check(s, 2, 10, F32, F32)


@pytest.mark.parametrize("rows", [2, 310])
@pytest.mark.parametrize("per_row", [255, 256, 257, 1000, 9001])
def test_long_bias_lists(rows, per_row):
    """Distinct tokens; in the last row one of them a second time, its first entry to be ignored."""
    _cuda()
    vocab = 9001
    s = settings(rows, vocab, seed=24, bias=0)
    g = np.random.default_rng(per_row)
    each = [g.permutation(vocab)[:per_row] for _ in range(rows)]
    each[-1] = np.append(each[-1], each[-1][per_row // 2])
    s["bias_tokens"] = np.concatenate(each).astype(np.int32)
    s["bias_values"] = g.normal(0, 5, s["bias_tokens"].size).astype(np.float32)
    s["bias_begin"] = np.cumsum([0] + [len(e) for e in each])
    check(s, rows, vocab, BF16, F32)


@pytest.mark.parametrize("tin,tout", PAIRS)
def test_special_values(tin, tout):
    """Infinities and NaN, in masked places and open ones; the type's lowest value; zeros of both signs."""
    _cuda()
    vocab = 2080
    x = torch.randn(6, vocab, device="cuda")
    for k, v in enumerate((np.nan, np.inf, -np.inf, torch.finfo(tin).min, torch.finfo(tin).max, 0.0, -0.0)):
        x[:, k::16] = v
    s = settings(6, vocab, history=400, seed=8)
    s["temperature"] = np.array([1, 2, 1, 0.5, np.nan, -1.0], np.float32)
    x[:, 3::16] /= 4  # stays finite under penalties and temperatures, where BF16 and 64 bits must not disagree
    x[:, 4::16] /= 4
    s["mask_row"] = np.array([-1, 1, 0, 2, 1, -1], np.int32)
    check(s, 6, vocab, tin, tout, x=x)


def test_rows_that_allow_nothing_and_everything():
    _cuda()
    vocab = 1000
    s = settings(4, vocab, seed=9)
    s["mask"] = np.stack([np.zeros(32, np.int32), np.full(32, -1, np.int32)])
    s["mask_row"] = np.array([0, 1, 0, -1], np.int32)
    x = torch.randn(4, vocab, device="cuda")
    x[0] = float("nan")
    y = plan_of(s, 4, vocab).shape(x)
    assert (y[0] == -float("inf")).all() and (y[2] == -float("inf")).all() and torch.isfinite(y[1]).all()
    d = plan_of(s, 4, vocab).backward(torch.full_like(x, float("nan")), logits=x)
    assert (d[0] == 0).all() and (d[2] == 0).all() and torch.isnan(d[1]).all()
    check(s, 4, vocab, BF16, F32)


def test_mask_without_rows_of_its_own_and_wide_masks():
    _cuda()
    s = settings(5, 100, seed=10)
    g = np.random.default_rng(0)
    s["mask"] = g.integers(-2 ** 31, 2 ** 31, (5, 9)).astype(np.int32)
    s["mask_row"] = None
    check(s, 5, 100, F32, F32)


@pytest.mark.parametrize("t", [F32, BF16])
def test_in_place(t):
    _cuda()
    rows, vocab = 5, 6007
    s = settings(rows, vocab, seed=11)
    plan = plan_of(s, rows, vocab)
    x = torch.randn(rows, vocab, device="cuda").to(t)
    y = plan.shape(x)
    z = x.clone()
    assert plan.shape(z, out=z) is z and torch.equal(y, z)
    d = torch.randn(rows, vocab, device="cuda").to(t)
    a = plan.backward(d, logits=x)
    b = d.clone()
    plan.backward(b, logits=x, out=b)
    assert torch.equal(a, b)
    # two column ranges of one matrix do not overlap
    both = torch.randn(rows, 2 * vocab, device="cuda").to(t)
    want = plan.shape(both[:, :vocab].contiguous())
    plan.shape(both[:, :vocab], out=both[:, vocab:])
    assert torch.equal(want, both[:, vocab:])


def test_decode_loop_updates_its_buffers():
    """New tokens appended between calls are seen; nothing is kept from the call before."""
    _cuda()
    vocab = 4000
    tokens = torch.zeros(64, dtype=torch.int32, device="cuda")
    begin = torch.tensor([0, 32], device="cuda")
    end = begin.clone()
    plan = pulse.LogitsPlan(2, vocab, tokens=tokens, begin=begin, end=end,
                            frequency=torch.tensor([1.0, 2.0], device="cuda"))
    x = torch.zeros(2, vocab, device="cuda")
    for k in range(20):
        y = plan.shape(x)
        want = torch.zeros(2, vocab, device="cuda")
        for r in range(2):
            for t in tokens[begin[r]:end[r]].tolist():
                want[r, t] -= r + 1
        assert torch.equal(y, want)
        new = torch.tensor([k % 3, 100 + k], dtype=torch.int32, device="cuda")
        tokens[end] = new
        end += 1
    # fewer rows than the plan has
    assert torch.equal(plan.shape(x[:1]), plan.shape(x)[:1])
    assert plan.shape(x[:0]).shape == (0, vocab)


def test_bad_indices_are_left_out_and_recorded():
    dev = _cuda()
    vocab = 300
    x = torch.randn(3, vocab, device="cuda")
    pulse.get_error(dev)

    def run(**kw):
        s = dict(NONE, repetition=np.full(3, 2.0, np.float32))
        s.update(kw)
        y = plan_of(s, 3, vocab).shape(x)
        assert pulse.get_error(dev) == pulse.pulse.PULSE_ERR_INDEX and pulse.get_error(dev) == 0
        plan_of(s, 3, vocab).backward(x, logits=x)
        pulse.get_error(dev)
        return y

    a = np.array
    y = run(tokens=a([5, vocab, -1, 2 ** 31 - 1], np.int32), begin=a([0, 0, 0]), end=a([4, 0, 1]))
    want, _ = ref.shape64(x.cpu().numpy(), dict(NONE, repetition=a([2.0] * 3), tokens=a([5]), begin=a([0, 0, 0]), end=a([1, 0, 1])))
    same(y, want, np.abs(want), F32)
    for begin, split, end in (([0, -1, 0], [0, 0, 0], [0, 1, 0]), ([0, 2, 0], [0, 2, 0], [0, 1, 0]),
                              ([0, 0, 0], [0, 0, 0], [0, 5, 0]), ([0, 0, 0], [0, 3, 0], [0, 2, 0]),
                              ([0, 1, 0], [0, 0, 0], [0, 2, 0])):
        y = run(tokens=a([1, 2, 3, 4], np.int32), begin=a(begin), split=a(split), end=a(end))
        assert torch.equal(y, x)
    y = run(bias_tokens=a([vocab, -5, 7], np.int32), bias_values=a([1, 1, 1], np.float32), bias_begin=a([0, 2, 3, 3]))
    want = x.clone()
    want[1, 7] += 1
    assert torch.equal(y, want)
    y = run(bias_tokens=a([1], np.int32), bias_values=a([1], np.float32), bias_begin=a([0, 2, 1, 1]))
    assert torch.equal(y, x)
    y = run(mask=np.zeros((2, 10), np.int32), mask_row=a([-1, 2, 1], np.int32))
    assert torch.equal(y[:2], x[:2]) and (y[2] == -float("inf")).all()


# Many CTAs' worth of rows, with two slices a row and more
@pytest.mark.parametrize("tin,tout", PAIRS)
@pytest.mark.parametrize("vocab", [16384, 20011, 24600])
def test_many_rows(tin, tout, vocab):
    _cuda()
    rows = 420
    check(settings(rows, vocab, history=60, seed=vocab, masks=7), rows, vocab, tin, tout)


@pytest.mark.parametrize("history", [1, 2047, 2048, 2049, 9000])
def test_many_rows_at_the_edges_of_blocks(history):
    """Histories that begin, split and end around block boundaries, and rows that share them."""
    _cuda()
    rows, vocab = 610, 8500
    g = np.random.default_rng(history)
    total = history + 4200
    s = settings(rows, vocab, seed=21, bias=3)
    s["tokens"] = np.minimum(np.exp(g.random(total) * np.log(vocab)).astype(np.int64) - 1, vocab - 1).clip(0).astype(np.int32)
    s["begin"] = g.integers(0, 4200, rows)
    s["begin"][:6] = [0, 2047, 2048, 2049, 4095, 4096]
    s["end"] = s["begin"] + history
    s["end"][7] = s["begin"][7]
    s["split"] = s["begin"] + (np.arange(rows) * 37) % (history + 1)
    s["split"][7] = s["begin"][7]
    check(s, rows, vocab, F32, F32)


def test_many_rows_of_one_sequence():
    _cuda()
    rows, vocab = 2300, 8300
    s = settings(rows, vocab, seed=22, bias=0)
    for k in ("bias_tokens", "bias_values", "bias_begin"):
        s[k] = None
    s["tokens"] = np.random.default_rng(1).integers(0, vocab, rows).astype(np.int32)
    s["begin"] = np.zeros(rows, np.int64)
    s["end"] = np.arange(rows)
    s["split"] = np.minimum(s["end"], 40)
    check(s, rows, vocab, BF16, BF16)


def test_many_rows_with_bad_indices():
    """Tokens outside the vocabulary count as an error only inside a row's history."""
    dev = _cuda()
    rows, vocab = 700, 9000
    tokens = np.random.default_rng(3).integers(0, vocab, 5000).astype(np.int32)
    tokens[[100, 2047, 2048]] = [-1, vocab, 2 ** 31 - 1]
    s = dict(NONE, tokens=tokens, repetition=np.full(rows, 2.0, np.float32), begin=np.full(rows, 101),
             end=np.full(rows, 2047))
    x = torch.randn(rows, vocab, device="cuda")
    pulse.get_error(dev)
    for begin, end, error in ((101, 2047, 0), (100, 200, 5), (2040, 2048, 5), (2048, 2049, 5), (2049, 5000, 0), (0, 5000, 5)):
        s["begin"], s["end"] = np.full(rows, 0), np.full(rows, 0)
        s["begin"][333], s["end"][333] = begin, end
        y = plan_of(s, rows, vocab).shape(x)
        assert pulse.get_error(dev) == error
        want, size = ref.shape64(x[333:334].cpu().numpy(), dict(s, begin=s["begin"][333:], end=s["end"][333:]))
        same(y[333:334], want, size, F32)
        assert torch.equal(y[:333], x[:333]) and torch.equal(y[334:], x[334:])


def test_many_rows_captured_in_a_graph():
    """Without a workspace (nothing is allocated in a capture) and with one."""
    _cuda()
    rows, vocab = 640, 8200
    s = settings(rows, vocab, seed=23)
    x = torch.randn(rows, vocab, device="cuda")
    plan = plan_of(s, rows, vocab)
    want = plan.shape(x)
    side = torch.cuda.Stream()
    for _ in range(2):
        out = torch.zeros_like(x)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                plan.shape(x, out=out)
            graph.replay()
            side.synchronize()
            assert torch.equal(out, want)
            plan.shape(x, out=out)  # allocates the stream's workspace
        side.synchronize()


# Long token lists are sorted by vocabulary slice first, in blocks of 2048 positions. The vocabulary
# here has 135 slices, so that some 130,000 tokens and 12 rows are enough.
WIDE = 1100000


@pytest.mark.parametrize("tin,tout", PAIRS)
@pytest.mark.parametrize("vocab", [WIDE, WIDE + 3])
@pytest.mark.parametrize("keys", [(), ("frequency", "presence", "bias_tokens", "bias_values", "bias_begin")])
def test_sorted_histories(tin, tout, vocab, keys):
    _cuda()
    s = settings(12, vocab, history=60000, seed=31, bias=40, **{k: None for k in keys})
    assert s["tokens"].size > 130000
    check(s, 12, vocab, tin, tout)


@pytest.mark.parametrize("history", [1, 2047, 2048, 2049, 9000, 100000])
def test_sorted_histories_at_the_edges_of_blocks(history):
    _cuda()
    rows = 12
    g = np.random.default_rng(history)
    total = 131072 + 4200
    s = settings(rows, WIDE, seed=32, bias=3)
    s["tokens"] = np.minimum(np.exp(g.random(total) * np.log(WIDE)).astype(np.int64) - 1, WIDE - 1).clip(0).astype(np.int32)
    s["begin"] = g.integers(0, 4200, rows)
    s["begin"][:8] = [0, 2047, 2048, 2049, 4095, 4096, total - history, total]
    s["end"] = s["begin"] + history
    s["end"][7] = s["begin"][7]
    s["split"] = s["begin"] + (np.arange(rows) * 37) % (history + 1)
    s["split"][7] = s["begin"][7]
    check(s, rows, WIDE, F32, F32)


def test_sorted_history_of_one_sequence():
    _cuda()
    rows, total = 12, 140000
    s = settings(rows, WIDE, seed=33)
    s["tokens"] = np.random.default_rng(1).integers(0, 5000, total).astype(np.int32)
    s["begin"] = np.zeros(rows, np.int64)
    s["end"] = np.arange(1, rows + 1) * (total // rows)
    s["split"] = np.minimum(s["end"], 20000)
    check(s, rows, WIDE, BF16, BF16)


def test_sorted_histories_with_bad_indices():
    dev = _cuda()
    rows = 12
    tokens = np.random.default_rng(3).integers(0, WIDE, 140000).astype(np.int32)
    tokens[[100, 2047, 2048]] = [-1, WIDE, 2 ** 31 - 1]
    s = dict(NONE, tokens=tokens, repetition=np.full(rows, 2.0, np.float32))
    x = torch.randn(rows, WIDE, device="cuda")
    pulse.get_error(dev)
    for begin, end, error in ((101, 2047, 0), (100, 200, 5), (2040, 2048, 5), (2048, 2049, 5), (2049, 140000, 0), (0, 5000, 5)):
        s["begin"], s["end"] = np.full(rows, 0), np.full(rows, 0)
        s["begin"][3], s["end"][3] = begin, end
        y = plan_of(s, rows, WIDE).shape(x)
        assert pulse.get_error(dev) == error
        want, size = ref.shape64(x[3:4].cpu().numpy(), dict(s, begin=s["begin"][3:], end=s["end"][3:]))
        same(y[3:4], want, size, F32)
        assert torch.equal(y[:3], x[:3]) and torch.equal(y[4:], x[4:])


def test_sorted_and_captured_calls_agree():
    """Nothing is sorted in a capture; the results have the same bits."""
    _cuda()
    rows = 12
    s = settings(rows, WIDE, history=60000, seed=34)
    x = torch.randn(rows, WIDE, device="cuda")
    d = torch.randn(rows, WIDE, device="cuda")
    plan = plan_of(s, rows, WIDE)
    want, back = plan.shape(x), plan.backward(d, logits=x)
    out, dx = torch.zeros_like(x), torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.shape(x, out=out)
            plan.backward(d, logits=x, out=dx)
        graph.replay()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(dx, back)


@pytest.mark.parametrize("rows,vocab,history", [(3, 5003, 60), (64, 32003, 500), (12, WIDE, 60000)])
def test_calls_back_to_back(rows, vocab, history):
    """Kernels start while the one in front of them ends: the bits are those of calls with a wait after each."""
    _cuda()
    s = settings(rows, vocab, history=history, seed=34)
    plan = plan_of(s, rows, vocab)
    tokens, bias = plan.tensors["tokens"], plan.tensors["bias_values"]
    first, first_bias = tokens.clone(), bias.clone()
    results = []
    for wait in (True, False):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        tokens.copy_(first), bias.copy_(first_bias)
        x = torch.randn(rows, vocab, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
        d, y, dx = (torch.zeros_like(x) for _ in range(3))
        seen = []
        for _ in range(20):
            x.mul_(0.9).add_(0.1)  # written by the kernel in front, as are the tokens and the biases
            tokens.add_(1).remainder_(vocab)
            bias.neg_()
            pause()
            plan.shape(x, out=y)
            pause()
            d.copy_(y).clamp_(-3, 3)
            pause()
            plan.backward(d, logits=x, out=dx)
            pause()
            x.add_(dx, alpha=0.01)  # read by the one behind
            seen.append(x[:, :: max(1, vocab // 997)].clone())
            pause()
        torch.cuda.synchronize()
        results.append(seen + [y.clone(), dx.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_on_another_stream():
    _cuda()
    rows, vocab = 16, 20011
    s = settings(rows, vocab, seed=12)
    plan = plan_of(s, rows, vocab)
    x = torch.randn(rows, vocab, device="cuda").to(BF16)
    want = plan.shape(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        z = x.clone()
        y = plan.shape(z, out_dtype=BF16)
    side.synchronize()
    assert torch.equal(y, want)


def test_offsets_past_32_bits():
    """The last rows of a logits buffer of more than 2^32 elements."""
    _cuda()
    rows, vocab, pitch = 5, 1001, (1 << 30) + 8
    x = torch.empty(4 * pitch + vocab, dtype=BF16, device="cuda")
    view = torch.as_strided(x, (rows, vocab), (pitch, 1))
    view.copy_(torch.randn(rows, vocab, device="cuda"))
    s = settings(rows, vocab, seed=13)
    y = plan_of(s, rows, vocab).shape(view, out_dtype=F32)
    want, size = ref.shape64(view.double().cpu().numpy(), s)
    same(y, want, size, F32)


def test_refusals():
    dev = _cuda()
    z = lambda *n, dt=F32: torch.zeros(*n, dtype=dt, device=dev)  # noqa: E731
    with pytest.raises(ValueError):
        pulse.LogitsPlan(3, 10, temperature=z(2))
    with pytest.raises(TypeError):
        pulse.LogitsPlan(3, 10, temperature=z(3, dt=torch.float64))
    with pytest.raises(TypeError):
        pulse.LogitsPlan(3, 10, tokens=z(3, dt=torch.int64), begin=z(3, dt=torch.int64), end=z(3, dt=torch.int64))
    with pytest.raises(ValueError):
        pulse.LogitsPlan(3, 100, mask=z(3, 3, dt=torch.int32))
    with pytest.raises(ValueError):
        pulse.LogitsPlan(3, 10, mask=z(2, 1, dt=torch.int32))
    with pytest.raises(ValueError):
        pulse.LogitsPlan(3, 40, mask=z(1, 2, dt=torch.int32).expand(3, 2))
    with pytest.raises(ValueError):
        pulse.LogitsPlan(3, 10, bias_tokens=z(4, dt=torch.int32), bias_values=z(3), bias_begin=z(4, dt=torch.int64))
    plan = pulse.LogitsPlan(3, 10, repetition=z(3) + 1, tokens=z(1, dt=torch.int32), begin=z(3, dt=torch.int64),
                            end=z(3, dt=torch.int64))
    for bad in (z(4, 10), z(3, 11), z(30), z(3, 20)[:, ::2]):
        with pytest.raises(ValueError):
            plan.shape(bad)
    with pytest.raises(TypeError):
        plan.shape(z(3, 10, dt=torch.float16))
    with pytest.raises(TypeError):
        plan.shape(z(3, 10), out_dtype=BF16)
    with pytest.raises(ValueError):
        plan.shape(z(3, 10), out=z(2, 10))
    x = z(3, 21)
    with pytest.raises(pulse.PulseError):
        plan.shape(x[:, :10], out=x[:, 5:15])
    with pytest.raises(pulse.PulseError):
        plan.shape(z(1, 10).expand(3, 10))
    with pytest.raises(ValueError):
        plan.backward(z(3, 10))
    with pytest.raises(TypeError):
        plan.backward(z(3, 10, dt=BF16), logits=z(3, 10))
    with pytest.raises(pulse.PulseError):
        plan.backward(z(3, 10), logits=x[:, :10], out=x[:, :10])
