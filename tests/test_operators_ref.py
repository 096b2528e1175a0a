"""CPU pins of the references of the optimizer step and the logit shaping: the
gradient against differences, the 8-bit codes against the definition, the
rounding's mean and the random bits' spread, and what 8-bit moments do to a
training run."""
import numpy as np
import pytest

import operators_ref as ref

RNG = np.random.default_rng


def test_mix_is_a_permutation_on_a_subset_and_spreads():
    x = np.arange(1 << 18, dtype=np.uint32)
    h = ref.mix(x)
    assert np.unique(h).size == x.size
    # every output bit is set half of the time: 4 sigma of 2^18 coins is 2^10
    for b in range(32):
        assert abs(int(((h >> np.uint32(b)) & 1).sum()) - (1 << 17)) < 1 << 10


def test_random_bits_depend_on_seed_step_block_and_place():
    a = ref.random_bits(0, 4096, 1, 1)
    for other in (ref.random_bits(0, 4096, 2, 1), ref.random_bits(0, 4096, 1, 2),
                  ref.random_bits(0, 4096, 1 << 32, 1), ref.random_bits(16, 4096, 1, 1)):
        assert (a == other).mean() < 0.01
    np.testing.assert_array_equal(ref.random_bits(0, 4096, 1, 1)[256:512], ref.random_bits(1, 256, 1, 1))
    # the halves that m and v take are not correlated: 5 sigma of 4096 samples
    lo, hi = (a & 0xFFFF) / 65536.0 - 0.5, (a >> 16) / 65536.0 - 0.5
    assert abs(np.mean(lo * hi)) * 12 < 5 / np.sqrt(a.size)


@pytest.mark.parametrize("signed", [True, False])
def test_codes_bracket_their_value_and_round_in_the_mean(signed):
    g = RNG(3)
    x = np.exp(g.normal(0, 2.0, 256)).astype(np.float32)
    if signed:
        x *= np.where(g.random(256) < 0.5, -1, 1).astype(np.float32)
    trials = 4000
    total = np.zeros(256)
    for k in range(trials):
        c, e = ref.encode8(x, g.integers(0, 65536, 256), signed)
        y = ref.decode8(c, e, signed)
        assert np.all(np.sign(y[y != 0]) == np.sign(x[y != 0]))
        step = np.abs(x) / 8 * (1 + 1e-6)
        # 14 binades under the block's maximum a first moment may fall to zero
        big = np.abs(x) > np.abs(x).max() * 2.0 ** -13
        assert np.all(np.abs(y - x)[big] <= step[big])
        total += y
    # mean of `trials` roundings of at most one step: 6 standard errors of a step / 2
    err = np.abs(total / trials - x)[big]
    assert np.all(err <= 6 * (np.abs(x) / 8 / 2)[big] / np.sqrt(trials))


def test_codes_at_the_edges():
    z = np.zeros(256, np.int64)
    f = np.full(256, 65535)
    # exact powers of two stay, whatever the random bits
    x = np.float32(2.0) ** -np.arange(256).clip(0, 13).astype(np.float32)
    for r in (z, f):
        np.testing.assert_array_equal(ref.decode8(*ref.encode8(x, r, True), True), x)
    # the largest value may round up past its binade
    x = np.full(256, np.float32(1.9999999))
    np.testing.assert_array_equal(ref.decode8(*ref.encode8(x, f, True), True), 2.0)
    np.testing.assert_array_equal(ref.decode8(*ref.encode8(x, z, True), True), 1.875)
    # a second moment above zero never becomes zero, a zero stays zero
    x = np.array([1.0, 1e-30, 1e-45, 0.0] * 64, np.float32)
    y = ref.decode8(*ref.encode8(x, z, False), False)
    assert (y[x > 0] > 0).all() and (y[x == 0] == 0).all()
    # a block with an infinity or NaN reads as NaN, its neighbour does not
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones(512, np.float32)
        x[17] = bad
        c, e = ref.encode8(x, np.zeros(512, np.int64), True)
        y = ref.decode8(c, e, True)
        assert np.isnan(y[:256]).all() and (y[256:] == 1).all() and e[0] == 0xFF and (c[:256] == 0x7F).all()
    # all-zero bytes are a state of zeros
    assert (ref.decode8(np.zeros(256, np.uint8), np.zeros(1, np.uint8), False) == 0).all()
    # tiny blocks: exponents are limited, values below FP32's normal range fall to the ends
    x = np.full(256, np.float32(1e-40))
    assert ref.encode8(x, z, True)[1][0] == 15 and ref.encode8(x, z, False)[1][0] == 31


def test_stochastic_codes_follow_a_slow_second_moment_and_nearest_ones_do_not():
    """beta2 = 0.999: a v that starts at a tenth of the squared gradient has to rise."""
    n, b2, steps = 256, 0.999, 3000
    start, target = np.full(n, 0.1, np.float32), 1.0
    true = target + (0.1 - target) * b2 ** steps
    ends = {}
    for kind in ("stochastic", "nearest"):
        c, e = ref.encode8(start, np.full(n, 32768), False)
        for t in range(1, steps + 1):
            v = ref.decode8(c, e, False).astype(np.float32)
            v = v * np.float32(b2) + np.float32(target) * np.float32(1 - b2)
            r = ref.random_bits(0, n, 5, t) & 0xFFFF if kind == "stochastic" else np.full(n, 32768)
            c, e = ref.encode8(v, r, False)
        ends[kind] = ref.decode8(c, e, False).mean()
    # a step is at most 1/8 of v; the walk's spread over 256 elements stays well inside 10 %
    assert abs(ends["stochastic"] / true - 1) < 0.1
    assert ends["nearest"] < 0.5 * true


def test_adam_first_step_moves_by_the_learning_rate():
    g = np.array([1.0, -2.0, 1e-3, 0.0])
    w, m, v = ref.adam64(np.zeros(4), g, np.zeros(4), np.zeros(4), 1, 1e-3, 0.9, 0.999, 1e-8)
    np.testing.assert_allclose(w, -1e-3 * np.sign(g) * [1, 1, 1 / (1 + 1e-5), 0], rtol=1e-6, atol=1e-15)


def test_moments_in_single_steps_follow_the_formula():
    g = RNG(1)
    x, m, v = (g.normal(0, 1e-3, 5000).astype(np.float32) for _ in range(3))
    v *= v
    m2, v2 = ref.moments32(x, m, v, 0.9, 0.999, 0.37)
    w, m3, v3 = ref.adam64(np.zeros(5000), x, m, v, 3, 1e-3, 0.9, 0.999, 1e-8, scale=float(np.float32(0.37)))
    # a sum of two products, five roundings with the constants' own
    assert np.all(np.abs(m2 - m3) <= 5 * 2.0 ** -24 * (0.9 * np.abs(m) + 0.1 * np.abs(0.37 * x)))
    assert np.all(np.abs(v2 - v3) <= 6 * 2.0 ** -24 * v3)
    w4, part = ref.weights64(np.zeros(5000), m3, v3, 3, 1e-3, 0.9, 0.999, 1e-8)
    np.testing.assert_allclose(w4, w, rtol=1e-12)


@pytest.mark.parametrize("seed", range(4))
def test_shaping_gradient_matches_differences(seed):
    g = RNG(seed)
    rows, vocab = 3, 37
    x = g.normal(0, 3, (rows, vocab))
    x[np.abs(x) < 1e-2] = 0.5  # away from the kink
    s = dict(tokens=g.integers(0, vocab, 60), begin=np.array([0, 20, 40]), split=np.array([5, 20, 60]),
             end=np.array([20, 40, 60]), repetition=np.array([1.3, 0.8, 1.1]), presence=np.array([.5, 0, -.2]),
             frequency=np.array([.1, .2, .3]), temperature=np.array([.7, 1.5, 0.0]),
             bias_tokens=np.array([3, 9, 3]), bias_values=np.array([1.0, -2.0, 4.0]), bias_begin=np.array([0, 3, 3, 3]),
             mask=g.integers(-2 ** 31, 2 ** 31, (2, 2)).astype(np.int32), mask_row=np.array([1, -1, 0]))
    d = g.normal(0, 1, (rows, vocab))

    def loss(z):
        y, _ = ref.shape64(z, s)
        return np.sum(d[np.isfinite(y)] * y[np.isfinite(y)])

    got = ref.shape64_backward(d, x, s)
    h = 1e-5
    for r in range(rows):
        for t in range(vocab):
            p, q = x.copy(), x.copy()
            p[r, t] += h
            q[r, t] -= h
            assert abs((loss(p) - loss(q)) / (2 * h) - got[r, t]) < 1e-7


def test_shaping_rows_that_allow_nothing():
    x = np.array([[np.nan, np.inf, 1.0], [1.0, 2.0, 3.0]])
    s = dict(mask=np.array([[0], [0b101]], np.int32))
    y, _ = ref.shape64(x, s)
    assert (y[0] == -np.inf).all() and y[1].tolist() == [1.0, -np.inf, 3.0]
    assert (ref.shape64_backward(np.full((2, 3), np.nan), x, s)[0] == 0).all()
