"""Plain references of the optimizer step and the logit shaping for the tests:
the formulas in float64, and the bit-level parts (moments rounded operation by
operation, 8-bit codes, random bits) in numpy integers. Shares no code with the
library."""
from __future__ import annotations

import numpy as np

BLOCK = 256
F32 = np.float32


# ------------------------------------------------------------------- AdamW

def adam64(w, g, m, v, step, lr, b1, b2, eps, wd=0.0, lr_scale=1.0, scale=1.0):
    """The whole step in float64: weights and moments."""
    w, g, m, v = (np.asarray(x, np.float64) for x in (w, g, m, v))
    g = g * scale
    rate = lr * lr_scale
    m2 = b1 * m + (1 - b1) * g
    v2 = b2 * v + (1 - b2) * g * g
    den = np.sqrt(v2 / (1 - b2 ** step)) + eps
    w2 = w - rate * (m2 / (1 - b1 ** step) / den + wd * w)
    return w2, m2, v2


def weights64(w, m2, v2, step, lr, b1, b2, eps, wd=0.0, lr_scale=1.0):
    """New weights in float64 from new moments as FP32 has them, and the size of the update's parts."""
    w, m2, v2 = (np.asarray(x, np.float64) for x in (w, m2, v2))
    with np.errstate(all="ignore"):
        a = lr * lr_scale * m2 / (1 - b1 ** step) / (np.sqrt(v2 / (1 - b2 ** step)) + eps)
        d = lr * lr_scale * wd * w
        return w - (a + d), np.abs(a) + np.abs(d)


def weight_tolerance(w2, part):
    """Half a unit in the last place of the result, and 16 units (2^-20) of the
    update's parts: 3 roundings of each of the two factors, 2 units each for square
    root and quotient and 2 roundings around them, 2 for the sums."""
    return np.abs(w2) * 2.0 ** -24 + part * 2.0 ** -20 + 1e-44


def moments32(g, m, v, b1, b2, scale=None):
    """FP32 moments, one rounding an operation."""
    g, m, v = (np.asarray(x, F32) for x in (g, m, v))
    with np.errstate(all="ignore"):
        if scale is not None:
            g = g * F32(scale)
        m2 = m * F32(b1) + g * F32(1.0 - b1)
        v2 = v * F32(b2) + (g * g) * F32(1.0 - b2)
    return m2, v2


def mix(x):
    x = np.asarray(x, np.uint32).copy()
    with np.errstate(over="ignore"):
        x ^= x >> np.uint32(16)
        x *= np.uint32(0xBB67AE85)
        x ^= x >> np.uint32(15)
        x *= np.uint32(0x9E3779B9)
        x ^= x >> np.uint32(16)
    return x


def random_bits(first_block, n, seed, step):
    """One uint32 per element of a tensor whose first block is `first_block`."""
    blocks = -(-n // BLOCK)
    gold = np.uint32(0x9E3779B9)
    with np.errstate(over="ignore"):
        key = np.zeros(1, np.uint32)
        for word in (seed & 0xFFFFFFFF, seed >> 32, step & 0xFFFFFFFF, step >> 32):
            key = mix(key + np.uint32(word) + gold)
        b = np.arange(first_block, first_block + blocks, dtype=np.uint64)
        low, high = (b & np.uint64(0xFFFFFFFF)).astype(np.uint32), (b >> np.uint64(32)).astype(np.uint32)
        key = mix(key ^ mix(low ^ mix(high)))
        h = mix(key[:, None] + np.arange(BLOCK, dtype=np.uint32)[None, :] * gold)
    return h.reshape(-1)[:n]


def _blocks(x):
    x = np.asarray(x)
    pad = -x.size % BLOCK
    return np.concatenate([x, np.zeros(pad, x.dtype)]).reshape(-1, BLOCK)


def encode8(x, r, signed):
    """(codes, exponents) of FP32 `x` with 16 random bits `r` an element."""
    n = np.asarray(x).size
    u = _blocks(np.asarray(x, F32)).view(np.uint32)
    mag = (u & np.uint32(0x7FFFFFFF)).astype(np.int64)
    top = mag.max(axis=1) >> 23
    under, low = (14, 15) if signed else (30, 31)
    e = np.clip(top, low, 253)
    c = ((mag + (_blocks(np.asarray(r, np.int64)) << 4)) >> 20) - 8 * (e - under)[:, None]
    c = np.clip(c, 0, 127 if signed else 255)
    if signed:
        c = c + 128 * (u >> np.uint32(31)).astype(np.int64)
    else:
        c = np.maximum(c, (mag > 0).astype(np.int64))
    bad = top == 255
    c[bad] = 0x7F
    e[bad] = 0xFF
    return c.astype(np.uint8).reshape(-1)[:n], e.astype(np.uint8)


def decode8(codes, e, signed):
    """float64 values of codes, from the definition of the format."""
    n = codes.size
    codes = _blocks(codes).astype(np.int64)
    c = codes % 128 if signed else codes
    exp = c // 8 + (e.astype(np.int64) - (14 if signed else 30))[:, None] - 127
    value = np.where(c > 0, (1 + (c % 8) / 8.0) * 2.0 ** exp.astype(np.float64), 0.0)
    if signed:
        value = np.where(codes >= 128, -value, value)
    value[e == 0xFF] = np.nan
    return value.reshape(-1)[:n]


# --------------------------------------------------------------- logits

def mask_bits(words, vocab):
    w = np.ascontiguousarray(words).view(np.uint32)
    t = np.arange(vocab)
    return (w[t >> 5] >> (t & 31).astype(np.uint32)) & 1 != 0


def _row(settings, key, r, other):
    return other if settings.get(key) is None else float(settings[key][r])


def _row_mask(s, r, vocab):
    if s.get("mask") is None:
        return None
    k = r if s.get("mask_row") is None else int(s["mask_row"][r])
    return None if k < 0 or k >= len(s["mask"]) else mask_bits(s["mask"][k], vocab)


def _history(s, r, vocab):
    """(seen, times generated) of row r; token numbers outside the vocabulary left out."""
    seen, count = np.zeros(vocab, bool), np.zeros(vocab)
    if s.get("tokens") is not None:
        b, e = int(s["begin"][r]), int(s["end"][r])
        m = b if s.get("split") is None else int(s["split"][r])
        for lo, hi, made in ((b, m, False), (m, e, True)):
            t = np.asarray(s["tokens"][lo:hi])
            t = t[(t >= 0) & (t < vocab)]
            seen[t] = True
            if made:
                np.add.at(count, t, 1.0)
    return seen, count


def shape64(x, s):
    """(y, size): float64 shaped rows and the size of the terms that made them."""
    x = np.asarray(x, np.float64)
    rows, vocab = x.shape
    y, size = np.empty_like(x), np.empty_like(x)
    with np.errstate(all="ignore"):
        for r in range(rows):
            seen, count = _history(s, r, vocab)
            rep, t = _row(s, "repetition", r, 1.0), _row(s, "temperature", r, 1.0)
            if not t > 0:
                t = 1.0
            a = np.where(seen, np.where(x[r] > 0, x[r] / rep, x[r] * rep), x[r])
            f, p = _row(s, "frequency", r, 0.0), _row(s, "presence", r, 0.0)
            b = np.zeros(vocab)
            if s.get("bias_tokens") is not None:
                lo, hi = int(s["bias_begin"][r]), int(s["bias_begin"][r + 1])
                for k in range(lo, hi):  # of a token listed twice, the last entry's value
                    if 0 <= int(s["bias_tokens"][k]) < vocab:
                        b[int(s["bias_tokens"][k])] = float(s["bias_values"][k])
            y[r] = (a - f * count - p * (count > 0) + b) / t
            size[r] = (np.abs(a) + abs(f) * count + abs(p) + np.abs(b)) / t
            ok = _row_mask(s, r, vocab)
            if ok is not None:
                y[r][~ok] = -np.inf
                size[r][~ok] = 0.0
    return y, size


def shape64_backward(d, x, s):
    d, x = np.asarray(d, np.float64), np.asarray(x, np.float64)
    out = np.empty_like(d)
    with np.errstate(all="ignore"):
        for r in range(d.shape[0]):
            seen, _ = _history(s, r, d.shape[1])
            rep, t = _row(s, "repetition", r, 1.0), _row(s, "temperature", r, 1.0)
            if not t > 0:
                t = 1.0
            out[r] = d[r] / t * np.where(seen, np.where(x[r] > 0, 1 / rep, rep), 1.0)
            ok = _row_mask(s, r, d.shape[1])
            if ok is not None:
                out[r][~ok] = 0.0
    return out
