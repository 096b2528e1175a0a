"""Optimizer step on the GPU against the float64 formulas and, for moments and
8-bit codes, bit for bit against numpy: ragged sizes, misaligned buffers, both
gradient types, missing gradients, skipped steps, non-finite values."""
import numpy as np
import pytest
import torch

import operators_ref as ref
import rl_post_trainer_gb300 as pulse
from pulse_testutil import Guarded

pytestmark = pytest.mark.gpu

SIZES = [1, 0, 5, 255, 256, 257, 4095, 4096, 4097, 8192, 12345, 70001, 7, 300]
LR, B1, B2, EPS = 1e-3, 0.9, 0.999, 1e-8


def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    return torch.device("cuda", 0)


class Shifted:
    """A guarded buffer whose usable part starts `shift` elements in."""

    def __init__(self, a, dtype, shift):
        self.box = Guarded(a.numel() + shift, dtype, "cuda")
        self.t = self.box.t[shift:]
        self.t.copy_(a.to(dtype))
        self.head = self.box.t[:shift].view(torch.uint8).clone()
        self.shift = shift

    def check(self):
        self.box.check()
        assert torch.equal(self.box.t[:self.shift].view(torch.uint8), self.head)


class Model:
    """Tensors of a plan and their numpy state."""

    def __init__(self, sizes, bits, grad=torch.float32, shift=0, seed=0, missing=(), scale=1e-3, codes=None):
        """codes: where the 8-bit codes start, if not where the others do."""
        g = torch.Generator().manual_seed(seed)
        self.bits, self.sizes, self.parts = bits, sizes, []
        self.wd = [0.01 if i % 2 else 0.0 for i in range(len(sizes))]
        self.ls = [(1.0, 0.5, 2.0)[i % 3] for i in range(len(sizes))]
        slots, first = [], 0
        for i, n in enumerate(sizes):
            p = {"n": n, "first": first, "buf": {}}
            first += -(-n // 256)
            size = torch.exp(2 * torch.randn(n, generator=g)) * scale
            grads = (torch.randn(n, generator=g) * size).to(grad)
            grads[torch.rand(n, generator=g) < 0.1] = 0
            w = torch.randn(n, generator=g) * 0.02
            m, v = torch.randn(n, generator=g) * size * 0.3, torch.rand(n, generator=g) * size * size
            v[torch.rand(n, generator=g) < 0.1] = 0
            p["g"], p["w"] = grads.float().numpy(), w.numpy()
            p["buf"]["w"] = Shifted(w, torch.float32, shift)
            p["buf"]["g"] = Shifted(grads, grad, shift)
            kw = {}
            if bits == 32:
                p["m"], p["v"] = m.numpy(), v.numpy()
                p["buf"]["m"], p["buf"]["v"] = Shifted(m, torch.float32, shift), Shifted(v, torch.float32, shift)
            else:
                for k, x, signed in (("m", m, True), ("v", v, False)):
                    c, e = ref.encode8(x.numpy(), np.full(n, 32768), signed)
                    p[k], p[k + "_exp"] = c, e
                    p["buf"][k] = Shifted(torch.from_numpy(c), torch.uint8, shift if codes is None else codes)
                    p["buf"][k + "_exp"] = Shifted(torch.from_numpy(e), torch.uint8, shift % 3)
                    p["buf"][k + "_out"] = Shifted(torch.zeros(n), torch.float32, shift)
                kw = {k: p["buf"][k].t for k in ("m_exp", "v_exp", "m_out", "v_out")}
            p["missing"] = i in missing
            slots.append(pulse.AdamTensorSlot(
                n, master=p["buf"]["w"].t, grad=None if p["missing"] else p["buf"]["g"].t, m=p["buf"]["m"].t,
                v=p["buf"]["v"].t, weight_decay=self.wd[i], lr_scale=self.ls[i], grad_dtype=grad, **kw))
            self.parts.append(p)
        self.plan = pulse.AdamPlan(slots, state_bits=bits)

    def step(self, t, scale=None, seed=0, lr=LR, b1=B1, b2=B2):
        s = None if scale is None else torch.tensor([scale], dtype=torch.float32, device="cuda")
        self.plan.step(t, lr, b1, b2, EPS, grad_scale=s, seed=seed)
        for i, p in enumerate(self.parts):
            if p["missing"] or (scale is not None and not np.isfinite(scale)):
                continue
            n = p["n"]
            with np.errstate(all="ignore"):
                if self.bits == 8:
                    m0 = ref.decode8(p["m"], p["m_exp"], True).astype(np.float32)
                    v0 = ref.decode8(p["v"], p["v_exp"], False).astype(np.float32)
                else:
                    m0, v0 = p["m"], p["v"]
                m, v = ref.moments32(p["g"], m0, v0, b1, b2, scale)
                w, part = ref.weights64(p["w"], m, v, t, lr, b1, b2, EPS, float(np.float32(self.wd[i])), self.ls[i])
            got = p["buf"]["w"].t.cpu().numpy()
            ok = np.isfinite(w)
            np.testing.assert_array_equal(np.isfinite(got), ok)
            assert np.all(np.abs(got - w)[ok] <= ref.weight_tolerance(w, part)[ok])
            p["w"] = got
            if self.bits == 32:
                p["m"], p["v"] = m, v
            else:
                r = ref.random_bits(p["first"], n, seed, t)
                p["m"], p["m_exp"] = ref.encode8(m, r >> np.uint32(16), True)
                p["v"], p["v_exp"] = ref.encode8(v, r & np.uint32(0xFFFF), False)

    def check(self):
        for p in self.parts:
            for k in ("m", "v") + (("m_exp", "v_exp") if self.bits == 8 else ()):
                np.testing.assert_array_equal(p["buf"][k].t.cpu().numpy(), p[k], err_msg=k)
            np.testing.assert_array_equal(p["buf"]["w"].t.cpu().numpy(), p["w"])
            for b in p["buf"].values():
                b.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 4, 8])
def test_ragged_model_over_steps(bits, grad, shift):
    _cuda()
    model = Model(SIZES, bits, grad, shift, seed=shift, missing=(3,))
    for t, scale in ((1, None), (2, 0.25), (3, 1.0), (1000, 0.7)):
        model.step(t, scale, seed=(t << 33) + 11)
        model.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 511, 1 << 20, 1000003])
def test_single_tensor(bits, n):
    _cuda()
    model = Model([n], bits, torch.bfloat16, seed=n)
    model.step(5, 0.5, seed=n)
    model.check()


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("total", [1200000, 1300021, 10000000, 10700009])
def test_eight_bit_plans_of_each_tile(total, shift, grad):
    """One, two and four blocks a warp on a GPU of 152 SMs, with the last tiles of the tensors cut anywhere."""
    _cuda()
    model = Model([total // 3 + 1, 777, total // 2, 256, total - total // 3 - total // 2], 8, grad, shift, seed=total,
                  codes=0)
    model.step(9, 0.5, seed=total << 3)
    model.plan.export_states()
    model.check()
    for p in model.parts:
        for k, signed in (("m", True), ("v", False)):
            out = p["buf"][k + "_out"].t.cpu().numpy()
            np.testing.assert_array_equal(out, ref.decode8(p[k], p[k + "_exp"], signed).astype(np.float32))


@pytest.mark.parametrize("bits", [32, 8])
def test_buffers_with_different_offsets(bits):
    """Weights, gradients and moments that no common offset aligns."""
    _cuda()
    n = 9001
    g = torch.Generator().manual_seed(1)
    for shifts in ((1, 0, 2, 3), (0, 1, 0, 0), (4, 0, 0, 4), (0, 4, 0, 0), (2, 2, 2, 1)):
        model = Model([n], bits, torch.bfloat16, 0, seed=3)
        p = model.parts[0]
        dt = torch.float32 if bits == 32 else torch.uint8
        for (k, d), s in zip((("w", torch.float32), ("g", torch.bfloat16), ("m", dt), ("v", dt)), shifts):
            p["buf"][k] = Shifted(p["buf"][k].t.clone(), d, s)
        kw = {k: p["buf"][k].t for k in ("m_exp", "v_exp", "m_out", "v_out")} if bits == 8 else {}
        model.plan = pulse.AdamPlan([pulse.AdamTensorSlot(n, p["buf"]["w"].t, p["buf"]["g"].t, p["buf"]["m"].t,
                                                          p["buf"]["v"].t, weight_decay=model.wd[0], lr_scale=model.ls[0], **kw)],
                                    state_bits=bits)
        model.step(2, 0.5, seed=9)
        model.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_scale_that_is_not_finite_skips(bits, scale):
    _cuda()
    model = Model(SIZES, bits, seed=2)
    model.step(3, scale)
    model.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38, 1e-30, 1e20, -0.0])
def test_special_gradients_stay_in_their_block(bits, value):
    _cuda()
    model = Model([1000, 600], bits, seed=4)
    p = model.parts[0]
    p["buf"]["g"].t[300] = value
    p["g"][300] = value
    for t in (1, 2):
        model.step(t, seed=t)
        model.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_all_zero(bits):
    """No gradient ever met: nothing moves but the decay, and nothing becomes NaN."""
    _cuda()
    n = 700
    z = torch.zeros(n, device="cuda")
    w = torch.ones(n, device="cuda")
    kw = {}
    if bits == 8:
        kw = {k: torch.zeros(pulse.adam_blocks(n), dtype=torch.uint8, device="cuda") for k in ("m_exp", "v_exp")}
    dt = torch.uint8 if bits == 8 else torch.float32
    m, v = torch.zeros(n, dtype=dt, device="cuda"), torch.zeros(n, dtype=dt, device="cuda")
    plan = pulse.AdamPlan([pulse.AdamTensorSlot(n, w, z, m, v, weight_decay=0.5, **kw)], state_bits=bits)
    plan.step(1, 0.25)
    assert torch.equal(w, torch.full_like(w, 0.875)) and not m.any() and not v.any()


@pytest.mark.parametrize("b1,b2", [(0.0, 0.0), (0.0, 0.999), (0.95, 0.95), (0.999, 0.9999)])
def test_betas(b1, b2):
    _cuda()
    for bits in (32, 8):
        model = Model([3001], bits, seed=6)
        for t in (1, 2, 77):
            model.step(t, None, 5, 3e-4, b1, b2)
            model.check()


def test_zero_learning_rate_moves_no_weight():
    _cuda()
    model = Model([3001], 32, seed=6)
    before = model.parts[0]["buf"]["w"].t.clone()
    model.step(1, lr=0.0)
    assert torch.equal(before, model.parts[0]["buf"]["w"].t)


def test_export_is_what_the_codes_stand_for():
    _cuda()
    for shift in (0, 1, 4):
        model = Model(SIZES, 8, seed=7, shift=shift)
        model.parts[4]["buf"]["g"].t[5] = float("nan")
        model.parts[4]["g"][5] = np.nan
        model.step(1, seed=1)
        model.plan.export_states()
        for p in model.parts:
            for k, signed in (("m", True), ("v", False)):
                want = ref.decode8(p[k], p[k + "_exp"], signed).astype(np.float32)
                np.testing.assert_array_equal(p["buf"][k + "_out"].t.cpu().numpy(), want)
        model.check()


def test_eight_bit_step_follows_the_thirty_two_bit_one():
    """Over 200 steps of noisy gradients the two optimizers move weights alike."""
    _cuda()
    n, g = 1 << 16, torch.Generator(device="cuda").manual_seed(3)
    mean = torch.randn(n, generator=g, device="cuda") * 1e-3
    w = {b: torch.zeros(n, device="cuda") for b in (32, 8)}
    grad = torch.empty(n, device="cuda")
    plans = {32: pulse.AdamPlan([pulse.AdamTensorSlot(n, w[32], grad, torch.zeros_like(mean), torch.zeros_like(mean))]),
             8: pulse.AdamPlan([pulse.AdamTensorSlot(n, w[8], grad, *(torch.zeros(k, dtype=torch.uint8, device="cuda")
                                                                      for k in (n, n, n // 256, n // 256)))], state_bits=8)}
    for t in range(1, 201):
        grad.copy_(mean + torch.randn(n, generator=g, device="cuda") * 1e-3)
        for p in plans.values():
            p.step(t, 1e-3, seed=17)
    a, b = w[32].double(), w[8].double()
    # a code step is 1/8: an update is off by a few per cent, unbiased, so 200 of them agree closely
    assert (torch.dot(a, b) / (a.norm() * b.norm())).item() > 0.995
    assert abs((b.norm() / a.norm()).item() - 1) < 0.05


@pytest.mark.parametrize("bits", [32, 8])
def test_same_bits_twice_and_on_another_stream(bits):
    _cuda()
    a, b = Model(SIZES, bits, seed=8, grad=torch.bfloat16), Model(SIZES, bits, seed=8, grad=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (1, 2, 3):
        a.plan.step(t, LR, seed=3)
        with torch.cuda.stream(side):
            b.plan.step(t, LR, seed=3)
    torch.cuda.synchronize()
    for p, q in zip(a.parts, b.parts):
        for k in p["buf"]:
            assert torch.equal(p["buf"][k].t, q["buf"][k].t)


def test_step_in_a_graph():
    _cuda()
    a, b = Model(SIZES, 8, seed=9), Model(SIZES, 8, seed=9)
    a.plan.step(4, LR, seed=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            norm, clip = b.plan.grad_norm(1e9)
            b.plan.step(4, LR, grad_scale=clip, seed=3)
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(a.parts, b.parts):
        assert torch.equal(p["buf"]["w"].t, q["buf"]["w"].t) and torch.equal(p["buf"]["m"].t, q["buf"]["m"].t)


def test_new_gradients():
    _cuda()
    model = Model([5000, 0, 300], 32, torch.bfloat16, seed=10)
    model.step(1)
    for k in range(3):
        g = [torch.randn(p["n"], device="cuda").to(torch.bfloat16) for p in model.parts]
        g[2] = None if k == 1 else g[2]
        model.plan.set_grads(g)
        for p, x in zip(model.parts, g):
            p["missing"] = x is None
            if x is not None:
                p["g"] = x.float().cpu().numpy()
        model.step(2 + k)
    model.check()
    with pytest.raises(ValueError):
        model.plan.set_grads([None])
    with pytest.raises(TypeError):
        model.plan.set_grads([torch.zeros(5000, device="cuda"), None, None])
    with pytest.raises(ValueError):
        model.plan.set_grads([torch.zeros(4999, device="cuda", dtype=torch.bfloat16), None, None])


# --------------------------------------------------------------------- norm

def _norm_plan(grads):
    return pulse.AdamPlan([pulse.AdamTensorSlot(g.numel(), grad=g) for g in grads], device=torch.device("cuda", 0))


# FP32 sums over at most 64 squares: 64 * 2^-24 relative at worst, halved by the root, and the result's rounding
NORM_TOL = 2.0 ** -19 + 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[1], [7], [255, 1, 0, 4096], [4097, 100003, 5], [1 << 20], [3333333, 17, 262144],
                                   [40000003, 1 << 20, 77, 60000001]])
def test_norm_and_clip(dtype, sizes):
    _cuda()
    gen = torch.Generator(device="cuda").manual_seed(len(sizes) + sizes[0])
    grads = []
    for i, n in enumerate(sizes):
        box = torch.randn(n + 3, generator=gen, device="cuda").to(dtype)
        grads.append(box[i % 4:i % 4 + n])
    want = np.sqrt(sum(float(np.square(g.double().cpu().numpy()).sum()) for g in grads))
    plan = _norm_plan(grads)
    for max_norm in (0.5 * want, 2 * want, 0.0, float("inf")):
        norm, clip = plan.grad_norm(float(np.float32(max_norm)))
        assert abs(norm.item() - want) <= want * NORM_TOL
        k = min(1.0, float(np.float32(max_norm)) / (want + 1e-6))
        assert abs(clip.item() - k) <= k * (NORM_TOL + 2.0 ** -22)
    again = plan.grad_norm(1.0)[0]
    assert torch.equal(norm, again)  # whatever the order in which CTAs finish


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_norm_that_is_not_finite(value):
    _cuda()
    g = torch.randn(100000, device="cuda")
    g[77777] = value
    norm, clip = _norm_plan([torch.ones(5, device="cuda"), g]).grad_norm(1.0)
    assert not np.isfinite(norm.item()) and np.isnan(clip.item())


def test_norm_of_nothing_and_of_zeros():
    _cuda()
    for grads in ([torch.zeros(0, device="cuda")], [torch.zeros(5000, device="cuda")]):
        norm, clip = _norm_plan(grads).grad_norm(1.0)
        assert norm.item() == 0.0 and clip.item() == 1.0
    plan = pulse.AdamPlan([pulse.AdamTensorSlot(5), pulse.AdamTensorSlot(2, grad=torch.full((2,), 3.0, device="cuda"))],
                          device=torch.device("cuda", 0))
    assert abs(plan.grad_norm(1.0)[0].item() - 18 ** 0.5) < 1e-6


def test_norm_into_given_outputs_and_small_values():
    _cuda()
    out, clip = Guarded(1, torch.float32), Guarded(1, torch.float32)
    g = torch.full((3000,), 1e-12, device="cuda")
    plan = _norm_plan([g])
    plan.grad_norm(1.0, out.t, clip.t)
    assert abs(out.t.item() - 1e-12 * 3000 ** 0.5) < 1e-15 and clip.t.item() == 1.0
    out.check(), clip.check()


def test_clipped_step_end_to_end():
    _cuda()
    model = Model([4000, 123], 32, torch.bfloat16, seed=12, scale=10.0)
    norm, clip = model.plan.grad_norm(1.0)
    assert norm.item() > 1.0 and 0 < clip.item() < 1.0
    model.step(1, float(clip.item()))
    model.check()


# ------------------------------------------------------------------ refusals

@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[300, 7, 70001], [1 << 20], [2000003, 4096, 400000]])
def test_calls_back_to_back(bits, sizes):
    """Kernels start while the one in front of them ends: the bits are those of calls with a wait after each."""
    _cuda()
    results = []
    for wait in (True, False):
        model = Model(sizes, bits, seed=5)
        grads = [p["buf"]["g"].t for p in model.parts]
        seen = []
        pause = torch.cuda.synchronize if wait else (lambda: None)
        for t in range(1, 41):
            for g in grads:
                g.mul_(-0.9).add_(1e-4)
            pause()
            norm, clip = model.plan.grad_norm(0.1)
            pause()
            model.plan.step(t, LR, B1, B2, EPS, grad_scale=clip, seed=t)
            pause()
            if bits == 8:
                model.plan.export_states()
                pause()
            seen += [norm, clip, model.parts[0]["buf"]["w"].t.sum(), model.parts[-1]["buf"]["w"].t.sum()]
            pause()
        torch.cuda.synchronize()
        names = ("w", "m", "v") + (("m_exp", "v_exp", "m_out", "v_out") if bits == 8 else ())
        results.append([x.clone() for x in seen] + [p["buf"][k].t.clone() for p in model.parts for k in names])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_refusals():
    dev = _cuda()
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device=dev)  # noqa: E731
    S = pulse.AdamTensorSlot
    with pytest.raises(ValueError):
        pulse.AdamPlan([S(8, f(7), f(8), f(8), f(8))])
    with pytest.raises(TypeError):
        pulse.AdamPlan([S(8, f(8), f(8), f(8, torch.uint8), f(8))])
    with pytest.raises(TypeError):
        pulse.AdamPlan([S(8, f(8), f(8), f(8), f(8))], state_bits=8)
    with pytest.raises(ValueError):
        pulse.AdamPlan([S(300, f(300), f(300), f(300, torch.uint8), f(300, torch.uint8), f(1, torch.uint8),
                          f(2, torch.uint8))], state_bits=8)
    with pytest.raises(TypeError):
        pulse.AdamPlan([S(8, f((8, 2))[:, 0], f(8), f(8), f(8))])
    with pytest.raises(pulse.PulseError):
        pulse.AdamPlan([S(8, f(8), f(8), f(8), f(8), weight_decay=-1.0)])
    norm_only = pulse.AdamPlan([S(8, grad=f(8))])
    with pytest.raises(pulse.PulseError):
        norm_only.step(1, 1e-3)
    with pytest.raises(pulse.PulseError):
        norm_only.export_states()
    with pytest.raises(pulse.PulseError):
        norm_only.grad_norm(-1.0)
    with pytest.raises(pulse.PulseError):
        norm_only.grad_norm(float("nan"))
    plan = pulse.AdamPlan([S(8, f(8), f(8), f(8), f(8))])
    with pytest.raises(pulse.PulseError):
        plan.export_states()
    with pytest.raises(ValueError):
        plan.step(0, 1e-3)
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=0.0),
                dict(eps=1e-40), dict(eps=float("inf"))):
        with pytest.raises(pulse.PulseError):
            plan.step(1, **{"lr": 1e-3, **bad})
    with pytest.raises(TypeError):
        plan.step(1, 1e-3, grad_scale=f(1, torch.float64))
    half = pulse.AdamPlan([S(8, f(8), f(8), f(8, torch.uint8), f(8, torch.uint8))], state_bits=8)
    with pytest.raises(pulse.PulseError):
        half.step(1, 1e-3)


# ------------------------------------------- gradients that move under a plan

def _new_grads(model, shift, seed):
    """Gradients for every tensor of the model, `shift` elements into their buffers."""
    gen = torch.Generator().manual_seed(seed)
    for p in model.parts:
        old = p["buf"]["g"].t
        g = (torch.randn(p["n"], generator=gen) * 1e-3).to(old.dtype)
        p["buf"]["g"], p["g"] = Shifted(g, old.dtype, shift), g.float().numpy()
    model.plan.set_grads([p["buf"]["g"].t for p in model.parts])


class Replayed:
    """A plan whose step is the replay of one captured step: its number, rate and seed stay."""

    def __init__(self, plan, t, seed):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        self.plan, self.graph, self.args = plan, torch.cuda.CUDAGraph(), (t, seed)
        with torch.cuda.stream(side), torch.cuda.graph(self.graph, stream=side):
            plan.step(t, LR, B1, B2, EPS, seed=seed)
        torch.cuda.current_stream().wait_stream(side)

    def step(self, t, lr, b1, b2, eps, grad_scale, seed):
        assert (t, seed) == self.args and grad_scale is None
        self.graph.replay()

    def set_grads(self, grads):
        self.plan.set_grads(grads)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("shifts", [(0, 1, 0, 4), (3, 0, 8, 2)])
def test_new_gradients_of_another_alignment(bits, grad, captured, shifts):
    """Gradients on their groups and off them in turn, also under a step that was captured with others."""
    _cuda()
    model = Model([70001, 256, 0, 5000, 8192], bits, grad, 0, seed=21)
    for k, shift in enumerate(shifts):
        _new_grads(model, shift, 100 + k)
        if captured and k == 0:
            model.plan = Replayed(model.plan, 5, 77)
        model.step(5, seed=77)
        model.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_new_gradients_in_a_capture_are_refused(bits):
    """The capture goes on, and the plan keeps the gradients it had."""
    _cuda()
    model = Model([3001, 40], bits, seed=22)
    other = [torch.ones(p["n"] + 1, device="cuda")[1:] for p in model.parts]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(2):  # without and with a staging buffer
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            with pytest.raises(pulse.PulseError):
                model.plan.set_grads(other)
            norm, clip = model.plan.grad_norm(1e30)
        torch.cuda.current_stream().wait_stream(side)
        graph.replay()
        want = np.sqrt(sum(float(np.square(p["g"].astype(np.float64)).sum()) for p in model.parts))
        assert abs(norm.item() - want) <= want * NORM_TOL and clip.item() == 1.0
        model.step(1 + k, seed=3)
        model.check()
        _new_grads(model, 1, 50 + k)


def test_misaligned_scalars_are_refused():
    """On the host, before any kernel sees them."""
    _cuda()
    import ctypes
    plan = Model([300], 32).plan
    lib, raw = pulse.lib(), torch.zeros(16, dtype=torch.uint8, device="cuda")
    at, invalid = raw.data_ptr(), pulse.pulse.PULSE_ERR_INVALID
    h = pulse.pulse.PulseAdamHyper(1, 0, LR, B1, B2, EPS)
    for off in (1, 2, 3):
        assert lib.pulse_grad_norm_multi(plan._h, 1.0, at + off, at + 4, None) == invalid
        assert lib.pulse_grad_norm_multi(plan._h, 1.0, at, at + 4 + off, None) == invalid
        assert lib.pulse_adam_step_multi(plan._h, ctypes.byref(h), at + off, None) == invalid
    assert not raw.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_of_tiny_gradients(dtype):
    """The small end of the norm's range: squares that are subnormal, and squares that are 0."""
    _cuda()
    n = 4096
    for power, want in ((-63, 2.0 ** -57), (-70, 2.0 ** -64), (-74, 2.0 ** -68), (-76, 0.0), (-100, 0.0)):
        norm, clip = _norm_plan([torch.full((n,), 2.0 ** power, dtype=dtype, device="cuda")]).grad_norm(1.0)
        assert norm.item() == want and clip.item() == 1.0  # sums of equal powers of 2 are exact
    g = (torch.rand(n + 5, device="cuda") * 1e-20).to(dtype)[5:]
    want = np.sqrt(np.square(g.double().cpu().numpy()).sum())
    # each of n squares is off by half of 2^-149, beside what larger gradients have
    tol = 0.5 * n * 2.0 ** -150 / want ** 2 + NORM_TOL
    assert abs(_norm_plan([g]).grad_norm(1.0)[0].item() - want) <= want * tol


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[33], [70001, 3, 8192], [5000011, 1 << 20]])
def test_norm_sums_of_32(dtype, sizes):
    """The documented accuracy: 32 squares in FP32, at most a rounding each, halved by the root, and two of the result."""
    _cuda()
    gen = torch.Generator(device="cuda").manual_seed(sizes[0])
    grads = [torch.randn(n, generator=gen, device="cuda").to(dtype) for n in sizes]
    want = np.sqrt(sum(float(np.square(g.double().cpu().numpy()).sum()) for g in grads))
    assert abs(_norm_plan(grads).grad_norm(1.0)[0].item() - want) <= want * (32 / 2 + 2) * 2.0 ** -24


@pytest.mark.parametrize("shift", [0, 1])
def test_second_moments_below_the_normal_range(shift):
    """FP32 moments: a subnormal v counts as it is under the root, beside an eps that is smaller still."""
    _cuda()
    n, eps = 3001, 2.0 ** -126
    model = Model([n], 32, shift=shift, seed=23)
    p = model.parts[0]
    g = torch.randn(n, generator=torch.Generator().manual_seed(1)) * 2.0 ** -66
    p["buf"]["g"].t.copy_(g)
    for k in ("m", "v"):
        p["buf"][k].t.zero_()
    model.plan.step(1, LR, 0.0, 0.0, eps)
    m, v = ref.moments32(g.numpy(), np.zeros(n), np.zeros(n), 0.0, 0.0)
    assert (v < 2.0 ** -126).all() and (v > 0).sum() > n // 2
    w, part = ref.weights64(p["w"], m, v, 1, LR, 0.0, 0.0, eps, float(np.float32(model.wd[0])), model.ls[0])
    got = p["buf"]["w"].t.cpu().numpy()
    assert np.all(np.abs(got - w) <= ref.weight_tolerance(w, part))
    np.testing.assert_array_equal(p["buf"]["v"].t.cpu().numpy(), v)
