"""Cases and plain forms of the trainer's optimizer step and the sampler's logit shaping.

Five operators, each in a plain form of elementary torch operations and as the
calls of the package:

* ``norm``   global gradient norm of many tensors and the clip factor
* ``adam32`` AdamW over many tensors, FP32 moments
* ``adam8``  AdamW over many tensors, 8-bit moments with a block exponent per
             256 elements, rounded stochastically; the moments are returned as
             the FP32 values they stand for
* ``shape``  penalties, biases, temperature and grammar masks on logits
* ``back``   the gradient of ``shape`` with respect to the raw logits

Tensors of one model live in one flat buffer per kind (weights, gradients,
moments), so outputs come back as those buffers. Vectors (norms, biases) follow
the matrices and take no weight decay.
"""
import math
import random

import torch

own = False

BLOCK = 256
LR, BETA1, BETA2, EPS, DECAY = 3e-6, 0.9, 0.999, 1e-8, 0.01
FIRST_STEP, RNG_SEED = 7, 0x5EED0123456789AB
KINDS = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # gradients of a small policy head: dozens of ragged tensors, latency counts
        {"name": "norm_ragged_small", "op": "norm", "layout": "split", "total": 1000003, "tensors": 37, "split": 11, "grad": "fp32"},
        # gradients of the whole 1.5B-parameter model set
        {"name": "norm_model_1.5b", "op": "norm", "layout": "model", "grad": "bf16"},
        # one tensor of 2^20 elements, the smallest configuration: launch latency
        {"name": "adam32_single_1m", "op": "adam32", "layout": "split", "total": 1 << 20, "tensors": 1, "split": 0, "grad": "fp32", "packed": False},
        # odd sizes back to back in one buffer, no tensor aligned to anything
        {"name": "adam32_packed_odd", "op": "adam32", "layout": "split", "total": 60000017, "tensors": 213, "split": 5, "grad": "bf16", "packed": True},
        # the whole 1.5B-parameter model set, BF16 gradients
        {"name": "adam32_model_1.5b", "op": "adam32", "layout": "model", "grad": "bf16", "packed": False},
        # adapters and heads of a few million parameters, 8-bit moments, odd sizes
        {"name": "adam8_ragged_3m", "op": "adam8", "layout": "split", "total": 3000017, "tensors": 61, "split": 3, "grad": "fp32"},
        # the whole 1.5B-parameter model set with 8-bit moments
        {"name": "adam8_model_1.5b", "op": "adam8", "layout": "model", "grad": "bf16"},
        # one request decoding: a single token's logits, everything switched on
        {"name": "shape_decode_1", "op": "shape", "rows": 1, "vocab": 151936, "in": "bf16", "out": "fp32", "history": 777, "train": False,
         "frequency": True, "bias": 40, "masked": 1.0},
        # a rollout batch with ragged histories, half of its rows under a grammar
        {"name": "shape_rollout_256", "op": "shape", "rows": 256, "vocab": 128256, "in": "bf16", "out": "bf16", "history": 8192, "train": False,
         "frequency": True, "bias": 100, "masked": 0.5},
        # log-probabilities of whole sequences on the trainer: row t sees the tokens before it; odd vocabulary
        {"name": "shape_train_odd", "op": "shape", "rows": 3001, "vocab": 32003, "in": "fp32", "out": "fp32", "history": 3001, "train": True,
         "frequency": False, "bias": 0, "masked": 0.0},
        # a handful of rows back from the loss
        {"name": "back_small", "op": "back", "rows": 5, "vocab": 32003, "in": "fp32", "out": "fp32", "history": 300, "train": False,
         "masked": 0.4},
        # the gradient of 4096 token positions in BF16
        {"name": "back_train_4096", "op": "back", "rows": 4096, "vocab": 151936, "in": "bf16", "out": "bf16", "history": 4096, "train": True,
         "masked": 0.25},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "adam32", "adam32", "adam8", "adam8", "shape", "shape", "shape", "back", "back"])
    if op in ("norm", "adam32", "adam8"):
        total = _log_uniform(rng, 5000, 1200000000)
        case = {"op": op, "layout": "split", "total": total, "tensors": min(_log_uniform(rng, 1, 400), max(1, total // 64)),
                "split": rng.randrange(1 << 20), "grad": rng.choice(["bf16", "fp32"])}
        if op == "adam32":
            case["packed"] = rng.random() < 0.4
        return case
    vocab = _log_uniform(rng, 1000, 200000)
    rows = _log_uniform(rng, 1, max(2, min(6000, 500000000 // vocab)))
    train = op == "back" or rng.random() < 0.3
    kind_in = rng.choice(["bf16", "fp32"])
    kind_out = "fp32" if kind_in == "fp32" else rng.choice(["bf16", "fp32"])
    history = rows if train else _log_uniform(rng, 1, min(32768, max(64, 8000000 // rows)))
    case = {"op": op, "rows": rows, "vocab": vocab, "in": kind_in, "out": kind_out, "history": history, "train": train,
            "masked": rng.choice([0.0, 0.3, 1.0])}
    if op == "shape":
        case.update({"frequency": rng.random() < 0.6, "bias": rng.choice([0, 0, 17, 300])})
    return case


def _sizes(case):
    """Element counts, matrices first, and how many of them are matrices."""
    if case["layout"] == "model":
        # 28 layers, hidden 1536, 12 query and 2 key/value heads of 128, MLP 8960, vocabulary 151936, tied embedding
        h, kv, mlp, layers = 1536, 256, 8960, 28
        layer = [h * h, kv * h, kv * h, h * h, mlp * h, mlp * h, h * mlp]
        matrices = [151936 * h] + layer * layers
        vectors = [h, kv, kv, h, h] * layers + [h]
        return matrices + vectors, len(matrices)
    rng = random.Random(case["split"] * 7919 + case["tensors"])
    k, total = case["tensors"], case["total"]
    weights = [math.exp(rng.uniform(0.0, 6.0)) for _ in range(k)]
    unit = (total - k) / sum(weights)
    sizes = [1 + int(w * unit) for w in weights]
    sizes[0] += total - sum(sizes)
    return sizes, k - k // 3


def _layout(case):
    """Offsets of the tensors in the flat buffer, its length, and where the vectors start."""
    sizes, matrices = _sizes(case)
    step = 1 if case.get("packed") else BLOCK
    offsets, at, edge = [], 0, 0
    for i, n in enumerate(sizes):
        if i == matrices:
            edge = at
        offsets.append(at)
        at += -(-n // step) * step
    return sizes, offsets, at, at if matrices == len(sizes) else edge


def work(case):
    op = case["op"]
    if op in ("norm", "adam32", "adam8"):
        n = sum(_sizes(case)[0])
        g = 2 if case["grad"] == "bf16" else 4
        if op == "norm":
            return {"bytes": n * g, "flops": 2 * n}
        if op == "adam32":
            return {"bytes": n * (24 + g), "flops": 16 * n}
        # the step (weights in and out, gradient, two code bytes in and out, two exponent bytes a block) and the FP32 values of the new moments
        return {"bytes": n * (8 + g + 4 + 8) + 4 * (n // BLOCK), "flops": 40 * n}
    size = {"bf16": 2, "fp32": 4}
    rows, vocab = case["rows"], case["vocab"]
    tokens = case["history"] if case["train"] else sum(_lengths(case))
    masks = _mask_rows(case) * ((vocab + 31) // 32) * 4
    bias = rows * case.get("bias", 0) * 8
    return {"bytes": rows * vocab * (size[case["in"]] + size[case["out"]]) + 4 * tokens + masks + bias, "flops": 4 * rows * vocab}


def _lengths(case):
    """History lengths of decoding rows: ragged up to case["history"], an empty one among several."""
    rng = random.Random(case["rows"] * 31 + case["history"])
    lens = [rng.randint(max(1, case["history"] // 4), case["history"]) for _ in range(case["rows"])]
    if len(lens) > 2:
        lens[1] = 0
    lens[-1] = case["history"]
    return lens


def _mask_rows(case):
    return int(round(case["masked"] * case["rows"]))


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] in ("norm", "adam32", "adam8"):
        return _prepare_optimizer(case, gen)
    return _prepare_logits(case, gen)


def _prepare_optimizer(case, gen):
    sizes, offsets, length, edge = _layout(case)
    s = {"op": case["op"], "edge": edge, "step": FIRST_STEP}
    grad = torch.randn(length, generator=gen, device=DEV)
    # gradients differ in size from place to place, and rows of an embedding that no token met get none
    scale = torch.exp(1.5 * torch.randn(-(-length // 4096), generator=gen, device=DEV)) * 1e-4
    scale[torch.rand(scale.numel(), generator=gen, device=DEV) < 0.05] = 0
    wide = scale.repeat_interleave(4096, output_size=scale.numel() * 4096)[:length]
    grad.mul_(wide)
    inside = None
    if sum(sizes) != length:  # nothing lives between the tensors
        inside = torch.zeros(length, dtype=torch.bool, device=DEV)
        for n, o in zip(sizes, offsets):
            inside[o:o + n] = True
        grad.mul_(inside)
    s["grad"] = grad.to(KINDS[case["grad"]])
    if case["op"] == "norm":
        s["max_norm"] = 1.0
    else:
        w = torch.randn(length, generator=gen, device=DEV).mul_(0.02)
        w[edge:] += 1.0
        m = torch.randn(length, generator=gen, device=DEV).mul_(0.3).mul_(wide)
        v = torch.rand(length, generator=gen, device=DEV).add_(0.05).mul_(wide).mul_(wide)
        if inside is not None:
            w.mul_(inside), m.mul_(inside), v.mul_(inside)
        s["w"] = w
        s["clip"] = torch.rand(1, generator=gen, device=DEV).mul_(0.5).add_(0.5)
        if case["op"] == "adam32":
            s["m"], s["v"] = m, v
        else:
            half = torch.full((), 0x8000, dtype=torch.int32, device=DEV)
            s["m"], s["m_exp"] = _encode8(m, half, 7)
            s["v"], s["v_exp"] = _encode8(v, half, 8)
            s["m_out"], s["v_out"] = torch.zeros_like(w), torch.zeros_like(w)
    del grad, wide, inside
    if own:
        import rl_post_trainer_gb300 as pulse
        slots = []
        for n, o in zip(sizes, offsets):
            part = {k: s[k][o:o + n] for k in ("grad", "w", "m", "v", "m_out", "v_out") if k in s}
            if case["op"] == "adam8":
                for k in ("m_exp", "v_exp"):
                    part[k] = s[k][o // BLOCK:o // BLOCK + -(-n // BLOCK)]
            slots.append(pulse.AdamTensorSlot(n, master=part.get("w"), grad=part["grad"], m=part.get("m"), v=part.get("v"),
                                              m_exp=part.get("m_exp"), v_exp=part.get("v_exp"), m_out=part.get("m_out"), v_out=part.get("v_out"),
                                              weight_decay=DECAY if o < edge else 0.0))
        s["plan"] = pulse.AdamPlan(slots, state_bits=8 if case["op"] == "adam8" else 32)
    return s


def _prepare_logits(case, gen):
    rows, vocab = case["rows"], case["vocab"]
    s = {"op": case["op"], "rows": rows, "vocab": vocab, "out_kind": KINDS[case["out"]]}
    s["logits"] = torch.randn(rows, vocab, generator=gen, device=DEV).mul_(4.0).to(KINDS[case["in"]])
    if case["train"]:  # one sequence: row t sees tokens [0, t), the first quarter of them the prompt
        tokens = case["history"]
        end = torch.arange(rows, device=DEV)
        begin = torch.zeros_like(end)
        split = torch.minimum(end, torch.full_like(end, tokens // 4))
        s["total"] = rows * (rows - 1) // 2
    else:
        lens = _lengths(case)
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        tokens = s["total"] = ends[-1]
        begin = torch.tensor(ends[:-1], device=DEV)
        end = torch.tensor(ends[1:], device=DEV)
        split = begin + (end - begin) // 3
    # words of a text: few of them often, most of them seldom
    u = torch.rand(max(tokens, 1), generator=gen, device=DEV, dtype=torch.float64)
    s["tokens"] = torch.exp(u * math.log(vocab)).to(torch.int32).sub_(1).clamp_(0, vocab - 1)
    s["begin"], s["split"], s["end"] = begin, split, end
    s["repetition"] = torch.rand(rows, generator=gen, device=DEV).mul_(0.4).add_(1.0)
    s["temperature"] = torch.rand(rows, generator=gen, device=DEV).add_(0.5)
    for key in ("presence", "frequency", "bias_tokens", "bias_values", "bias_begin", "mask", "mask_row"):
        s[key] = None
    if case.get("frequency"):
        s["presence"] = torch.rand(rows, generator=gen, device=DEV).mul_(0.6)
        s["frequency"] = torch.rand(rows, generator=gen, device=DEV).mul_(0.3)
    if case.get("bias"):
        k = min(case["bias"], vocab)
        start = torch.randint(vocab, (rows, 1), generator=gen, device=DEV)
        apart = max(1, vocab // k)
        s["bias_tokens"] = ((start + apart * torch.arange(k, device=DEV)) % vocab).to(torch.int32).reshape(-1).contiguous()
        s["bias_values"] = torch.randn(rows * k, generator=gen, device=DEV).mul_(3.0)
        s["bias_begin"] = torch.arange(rows + 1, device=DEV) * k
    masks = _mask_rows(case)
    if masks:  # grammar states that allow a few per cent of the tokens, and one that allows none
        words = (vocab + 31) // 32
        a, b, c = (torch.randint(-2 ** 31, 2 ** 31, (masks, words), generator=gen, device=DEV, dtype=torch.int64).to(torch.int32) for _ in range(3))
        s["mask"] = a & b & c
        if masks > 2:
            s["mask"][1] = 0
        who = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
        who[torch.randperm(rows, generator=gen, device=DEV)[:masks]] = torch.arange(masks, dtype=torch.int32, device=DEV)
        s["mask_row"] = who
    if case["op"] == "back":
        s["dout"] = torch.randn(rows, vocab, generator=gen, device=DEV).mul_(1e-3).to(KINDS[case["out"]])
        s["din"] = torch.empty_like(s["logits"])
    else:
        s["out"] = torch.empty(rows, vocab, dtype=KINDS[case["out"]], device=DEV)
    if own:
        import rl_post_trainer_gb300 as pulse
        s["plan"] = pulse.LogitsPlan(rows, vocab, device=s["logits"].device, **{k: s[k] for k in (
            "tokens", "begin", "split", "end", "repetition", "presence", "frequency", "temperature",
            "bias_tokens", "bias_values", "bias_begin", "mask", "mask_row")})
    return s


# ------------------------------------------------------------- the operators

def run(s):
    op = s["op"]
    if op == "norm":
        if own:
            norm, clip = s["plan"].grad_norm(s["max_norm"])
        else:
            norm = torch.sqrt(torch.sum(torch.square(s["grad"].float()))).reshape(1)
            clip = torch.where(torch.isfinite(norm), torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0), math.nan)
        return {"norm": norm, "clip": clip}
    if op == "adam32":
        if own:
            s["plan"].step(s["step"], LR, BETA1, BETA2, EPS, grad_scale=s["clip"])
        else:
            m, v, w = _adam(s, s["m"], s["v"])
            s["m"].copy_(m), s["v"].copy_(v), s["w"].copy_(w)
        s["step"] += 1
        return {"w": s["w"], "m": s["m"], "v": s["v"]}
    if op == "adam8":
        if own:
            s["plan"].step(s["step"], LR, BETA1, BETA2, EPS, grad_scale=s["clip"], seed=RNG_SEED)
            s["plan"].export_states()
        else:
            m, v, w = _adam(s, _decode8(s["m"], s["m_exp"], 7), _decode8(s["v"], s["v_exp"], 8))
            s["w"].copy_(w)
            bits = _random_bits(w.numel(), s["step"])
            s["m"], s["m_exp"] = _encode8(m, bits >> 16, 7)
            s["v"], s["v_exp"] = _encode8(v, bits & 0xFFFF, 8)
            s["m_out"] = _decode8(s["m"], s["m_exp"], 7)
            s["v_out"] = _decode8(s["v"], s["v_exp"], 8)
        s["step"] += 1
        return {"w": s["w"], "m": s["m_out"], "v": s["v_out"]}
    if op == "shape":
        if own:
            return s["plan"].shape(s["logits"], out=s["out"])
        return _shape(s).to(s["out_kind"])
    if own:
        return s["plan"].backward(s["dout"], logits=s["logits"], out=s["din"])
    return _back(s)


def _adam(s, m, v):
    """New moments and weights, one rounding to FP32 an operation."""
    t, w = s["step"], s["w"]
    g = s["grad"].float() * s["clip"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    u = m / (torch.sqrt(v) * (1.0 / math.sqrt(1.0 - BETA2 ** t)) + EPS) * (LR / (1.0 - BETA1 ** t))
    u[:s["edge"]] += w[:s["edge"]] * (LR * DECAY)
    return m, v, w - u


# 8-bit moments: a code holds an exponent and three mantissa bits, counted from a base that the block's largest exponent sets.

def _base(exp, bits):
    """First FP32 exponent field of the codes, times 8: 16 binades of 7-bit codes, 32 of 8-bit ones, one of them above the block's maximum."""
    return (exp.to(torch.int32) - (14 if bits == 7 else 30)) * 8


def _decode8(codes, exp, bits):
    c = codes.to(torch.int32).reshape(-1, BLOCK)
    low = c & ((1 << bits) - 1)
    value = ((low + _base(exp, bits)[:, None]) << 20).view(torch.float32)
    value = torch.where(low == 0, 0.0, value)
    return (torch.where(c > 127, -value, value) if bits == 7 else value).reshape(-1)


def _encode8(x, r, bits):
    """Codes and block exponents; r: 16 random bits an element, which round the dropped part of the mantissa."""
    raw = x.view(torch.int32).reshape(-1, BLOCK)
    mag = raw & 0x7FFFFFFF
    exp = torch.clamp(torch.amax(mag, 1) >> 23, 15 if bits == 7 else 31, 253)
    r = r.to(torch.int32)
    c = ((mag + ((r if r.dim() == 0 else r.reshape(-1, BLOCK)) << 4)) >> 20) - _base(exp, bits)[:, None]
    c = torch.clamp(c, 0, (1 << bits) - 1)
    # a second moment above zero stays above zero, a first moment keeps its sign
    c = torch.where(raw < 0, c + 128, c) if bits == 7 else torch.maximum(c, (mag > 0).to(torch.int32))
    return c.to(torch.uint8).reshape(-1), exp.to(torch.uint8)


def _mix(x):
    """A 32-bit hash of whole numbers held in 64 bits."""
    x = ((x ^ (x >> 16)) * 0xBB67AE85) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x9E3779B9) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_bits(n, step):
    """32 random bits an element: a hash of seed, step, block and place in the block."""
    key = 0
    for word in (RNG_SEED & 0xFFFFFFFF, RNG_SEED >> 32, step & 0xFFFFFFFF, step >> 32):
        key = _mix((key + word + 0x9E3779B9) & 0xFFFFFFFF)
    block = torch.arange(n // BLOCK, device=DEV, dtype=torch.int64)
    key = _mix((key ^ _mix((block & 0xFFFFFFFF) ^ _mix(block >> 32))) & 0xFFFFFFFF)
    place = torch.arange(BLOCK, device=DEV, dtype=torch.int64) * 0x9E3779B9
    return _mix((key[:, None] + place[None, :]) & 0xFFFFFFFF).reshape(-1)


def _history(s):
    """Row and token of every history entry, and whether it was generated."""
    rows, lens = s["rows"], s["end"] - s["begin"]
    row = torch.repeat_interleave(torch.arange(rows, device=DEV), lens, output_size=s["total"])
    first = torch.cumsum(lens, 0) - lens
    at = torch.arange(s["total"], device=DEV) - first[row] + s["begin"][row]
    return row * s["vocab"] + s["tokens"][at].long(), at >= s["split"][row]


def _allowed(s):
    words = s["mask"][s["mask_row"].clamp(min=0).long()]
    bits = (words[:, :, None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
    return (bits.reshape(s["rows"], -1)[:, :s["vocab"]] != 0) | (s["mask_row"] < 0)[:, None]


def _shape(s):
    x = s["logits"].float()
    key, generated = _history(s)
    seen = torch.zeros(x.numel(), dtype=torch.bool, device=DEV)
    seen[key] = True
    r = s["repetition"][:, None]
    x = torch.where(seen.reshape(x.shape), torch.where(x > 0, x / r, x * r), x)
    if s["frequency"] is not None:
        count = torch.zeros(x.numel(), device=DEV).index_add_(0, key, generated.float()).reshape(x.shape)
        x = x - s["frequency"][:, None] * count
        x = x - s["presence"][:, None] * (count > 0)
    if s["bias_tokens"] is not None:
        row = torch.arange(s["rows"], device=DEV).repeat_interleave(s["bias_tokens"].numel() // s["rows"])
        x.view(-1).index_add_(0, row * s["vocab"] + s["bias_tokens"].long(), s["bias_values"])
    x = x * (1.0 / s["temperature"])[:, None]
    return x if s["mask"] is None else torch.where(_allowed(s), x, -math.inf)


def _back(s):
    d = s["dout"].float() * (1.0 / s["temperature"])[:, None]
    key, _ = _history(s)
    seen = torch.zeros(d.numel(), dtype=torch.bool, device=DEV)
    seen[key] = True
    r = s["repetition"][:, None]
    d = torch.where(seen.reshape(d.shape), torch.where(s["logits"] > 0, d / r, d * r), d)
    if s["mask"] is not None:
        d = torch.where(_allowed(s), d, 0.0)
    return d.to(s["logits"].dtype)


# --------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        if case["op"] == "norm":
            return _exact_norm(s)
        if case["op"] in ("adam32", "adam8"):
            return _exact_adam(s, case["op"] == "adam8")
        return _exact_logits(s, case)


def _exact_norm(s):
    g = s.pop("grad").double()
    norm = torch.linalg.vector_norm(g).item()
    return {"norm": torch.tensor([norm], dtype=torch.float64), "clip": torch.tensor([min(1.0, s["max_norm"] / (norm + 1e-6))], dtype=torch.float64)}


def _exact_adam(s, eight):
    t, w = s["step"], s["w"].double()
    g = s.pop("grad").double() * s["clip"].double()
    m, v = (_exact_values(s, k) if eight else s.pop(k).double() for k in ("m", "v"))
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    del g
    u = (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    u[:s["edge"]] += DECAY * w[:s["edge"]]
    w -= LR * u
    del u
    if eight:
        bits = _exact_bits(w.numel() // BLOCK, t)
        m = _exact_rounded(m, bits // 65536, 14, 127)
        v = _exact_rounded(v, bits % 65536, 30, 255)
    return {"w": w, "m": m, "v": v}


def _exact_values(s, k):
    codes, exp = s.pop(k).reshape(-1, BLOCK), s.pop(k + "_exp")
    low = (codes % 128 if k == "m" else codes).double()
    power = torch.floor(low / 8) + (exp.double() - (14 if k == "m" else 30) - 127)[:, None]
    value = torch.ldexp(1 + torch.remainder(low, 8) / 8, power) * (low > 0)
    return (value * (1 - 2.0 * (codes // 128)) if k == "m" else value).reshape(-1)


def _exact_rounded(x, r, under, most):
    """x to three mantissa bits between `under` binades below its block's and one above, up where the dropped part and r / 65536 sum to 1."""
    x = x.reshape(-1, BLOCK)
    a = x.abs()
    _, top = torch.frexp(a.amax(1))
    top = torch.clamp(top.double() - 1, min=(under + 1) - 127)
    f, e = torch.frexp(a)
    place = 8 * (e.double() - 1 - (top - under)[:, None]) + 8 * (2 * f - 1)
    del f, e
    c = torch.clamp(torch.floor(place + r.reshape(-1, BLOCK) / 65536), 0, most)
    c = torch.where((c == 0) & (a > 0) & (most == 255), 1.0, c)
    c = torch.where(a == 0, 0.0, c)
    value = torch.ldexp(1 + torch.remainder(c, 8) / 8, torch.floor(c / 8) + (top - under)[:, None]) * (c > 0)
    return torch.where(x < 0, -value, value).reshape(-1)


def _exact_bits(blocks, step):
    def stir(a):  # on whole numbers, 32 bits of them
        a = (a ^ (a // 65536)) * 3144134277 % 4294967296
        a = (a ^ (a // 32768)) * 2654435769 % 4294967296
        return a ^ (a // 65536)
    key = 0
    for part in (RNG_SEED % 2 ** 32, RNG_SEED // 2 ** 32, step, 0):
        key = stir((key + part + 2654435769) % 2 ** 32)
    block = torch.arange(blocks, device=DEV)
    key = stir(stir(block ^ stir(0)) ^ key)
    return stir((key.unsqueeze(1) + 2654435769 * torch.arange(BLOCK, device=DEV)) % 2 ** 32).reshape(-1)


def _exact_logits(s, case):
    rows, vocab = s["rows"], s["vocab"]
    begin, split, end = (s[k].tolist() for k in ("begin", "split", "end"))
    raw = s.pop("logits").double()
    out = s["dout"].double() if case["op"] == "back" else raw
    words = torch.arange(vocab, device=DEV)
    answer = torch.empty(rows, vocab, dtype=torch.float64, device=DEV)
    for i in range(rows):
        counts = torch.bincount(s["tokens"][split[i]:end[i]], minlength=vocab)
        before = torch.bincount(s["tokens"][begin[i]:split[i]], minlength=vocab)
        r, t = s["repetition"][i].double(), s["temperature"][i].double()
        pull = torch.where((counts + before > 0), torch.where(raw[i] > 0, 1 / r, r), torch.ones_like(r))
        y = out[i] * pull
        if case["op"] == "shape":
            if s["frequency"] is not None:
                y = y - s["frequency"][i].double() * counts - s["presence"][i].double() * (counts > 0)
            if s["bias_tokens"] is not None:
                a, b = (int(k) for k in s["bias_begin"][i:i + 2])
                y[s["bias_tokens"][a:b].long()] += s["bias_values"][a:b].double()
        y = y / t
        if s["mask"] is not None and int(s["mask_row"][i]) >= 0:
            bits = (s["mask"][int(s["mask_row"][i])].long() % 2 ** 32)[words // 32]
            shut = (bits >> (words % 32)) % 2 == 0
            y[shut] = -math.inf if case["op"] == "shape" else 0.0
        answer[i] = y
    return answer
