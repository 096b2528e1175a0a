"""One reinforcement-learning loop on one GPU, from the rollout to the served weights.

    python examples/rollout_and_step.py [--iterations 30] [--state-bits 8]

A toy policy (an embedding and an output matrix) writes sequences under the
settings a serving engine would apply (penalties, a temperature, a grammar), is
rewarded for tokens of one kind, and learns:

1. sampler: BF16 weights -> logits -> LogitsPlan.shape -> a token per sequence,
   appended to the plan's own token buffer
2. trainer: the logits of every position at once, shaped by the same settings with
   the tokens before it as its history -> policy gradient -> LogitsPlan.backward
3. AdamPlan.grad_norm -> AdamPlan.step, clipped on the device
4. Plan.encode: the BF16 patch of what the step moved -> Plan.apply on the sampler

At the end of every iteration the sampler's weights equal the trainer's BF16 view
bit for bit. Logits of the same bits are shaped to the same bits by the sampler's plan
and the trainer's; the log-probabilities that the two see differ only where a last bit
of a BF16 logit does, their matrix products being of different heights.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import rl_post_trainer_gb300 as pulse  # noqa: E402

VOCAB, HIDDEN, SEQUENCES, PROMPT, LENGTH = 1003, 64, 48, 4, 20


class Trainer:
    """FP32 master weights, their BF16 view and patch buffers, gradients and moments."""

    def __init__(self, state_bits: int, gen: torch.Generator):
        dev = torch.device("cuda", 0)
        self.weights = [torch.randn(VOCAB, HIDDEN, generator=gen, device=dev) * 0.3 for _ in range(2)]
        self.grads = [torch.zeros_like(w) for w in self.weights]
        self.views = [w.to(torch.bfloat16) for w in self.weights]
        self.idx = [torch.empty(w.numel(), dtype=torch.int32, device=dev) for w in self.weights]
        self.val = [torch.empty(w.numel(), dtype=torch.bfloat16, device=dev) for w in self.weights]
        moment = torch.uint8 if state_bits == 8 else torch.float32
        slots = []
        for w, g in zip(self.weights, self.grads):
            n = w.numel()
            m, v = (torch.zeros(n, dtype=moment, device=dev) for _ in range(2))
            exps = {k: torch.zeros(pulse.adam_blocks(n), dtype=torch.uint8, device=dev)
                    for k in ("m_exp", "v_exp")} if state_bits == 8 else {}
            slots.append(pulse.AdamTensorSlot(n, master=w.view(-1), grad=g.view(-1), m=m, v=v, weight_decay=0.01, **exps))
        self.adam = pulse.AdamPlan(slots, state_bits=state_bits)
        self.encode = pulse.Plan([pulse.TensorSlot(w.numel(), master=w.view(-1), prev=p.view(-1), idx=i, val=v)
                                  for w, p, i, v in zip(self.weights, self.views, self.idx, self.val)]).encode


class Sampler:
    """The served BF16 weights, patched in place."""

    def __init__(self, trainer: Trainer):
        self.weights = [p.clone() for p in trainer.views]
        self.apply = pulse.Plan([pulse.TensorSlot(w.numel(), w=w.view(-1), idx=i, val=v)
                                 for w, i, v in zip(self.weights, trainer.idx, trainer.val)]).apply


def logits_of(weights, tokens: torch.Tensor) -> torch.Tensor:
    return weights[0][tokens.long()] @ weights[1].t()


def plans(tokens: torch.Tensor):
    """The sampler's plan (a row a sequence, its history up to `end`) and the trainer's (a row a
    generated position, in the order of the sequences), with the same settings; `split`, `end`."""
    dev, total = tokens.device, tokens.shape[1]
    begin = torch.arange(SEQUENCES, device=dev) * total
    split, end = begin + PROMPT, begin + PROMPT
    settings = {"repetition": 1.05, "presence": 0.1, "frequency": 0.05, "temperature": 0.9}
    # a grammar that forbids every seventh token to every second sequence
    allowed = torch.arange(VOCAB, device=dev) % 7 != 0
    bits = torch.zeros((VOCAB + 31) // 32 * 32, dtype=torch.int64, device=dev)
    bits[:VOCAB] = allowed
    words = (bits.view(-1, 32) << torch.arange(32, device=dev)).sum(1)
    mask = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32).view(1, -1)
    mask_row = torch.arange(SEQUENCES, device=dev, dtype=torch.int32) % 2 - 1  # -1: none

    def plan(rows_of_sequence, begin, split, end):
        n = SEQUENCES * rows_of_sequence
        each = {k: torch.full((n,), v, device=dev) for k, v in settings.items()}
        return pulse.LogitsPlan(n, VOCAB, tokens=tokens.view(-1), begin=begin, split=split, end=end, mask=mask,
                                mask_row=mask_row.repeat_interleave(rows_of_sequence), **each)

    decode = plan(1, begin, split, end)
    step = torch.arange(LENGTH, device=dev).repeat(SEQUENCES)
    wide = [t.repeat_interleave(LENGTH) for t in (begin, split)]
    return decode, plan(LENGTH, wide[0], wide[1], wide[1] + step), split, end


def run(iterations: int = 30, state_bits: int = 8, seed: int = 0, lr: float = 0.1):
    """Mean reward of every iteration, and the largest difference of log-probabilities."""
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(seed)
    trainer = Trainer(state_bits, gen)
    sampler = Sampler(trainer)

    tokens = torch.zeros(SEQUENCES, PROMPT + LENGTH, dtype=torch.int32, device=dev)
    decode, train, split, end = plans(tokens)

    rewards, apart = [], 0.0
    for iteration in range(1, iterations + 1):
        # rollout: the token buffer and `end` move under the plan
        tokens[:, :PROMPT] = torch.randint(1, VOCAB, (SEQUENCES, PROMPT), generator=gen, device=dev, dtype=torch.int32)
        seen = torch.empty(SEQUENCES, LENGTH, device=dev)
        for t in range(LENGTH):
            end.copy_(split + t)
            shaped = decode.shape(logits_of(sampler.weights, tokens[:, PROMPT + t - 1]), out_dtype=torch.float32)
            logp = torch.log_softmax(shaped, -1)
            new = torch.multinomial(logp.exp(), 1, generator=gen)
            tokens[:, PROMPT + t] = new[:, 0].to(torch.int32)
            seen[:, t] = logp.gather(1, new)[:, 0]
        chosen = tokens[:, PROMPT:].long()
        reward = (chosen % 5 == 0).float()
        rewards.append(reward.mean().item())

        # policy gradient at the distribution that the tokens were drawn from
        before = tokens[:, PROMPT - 1:-1].reshape(-1)
        raw = logits_of(trainer.views, before)
        logp = torch.log_softmax(train.shape(raw, out_dtype=torch.float32), -1)
        taken = logp.gather(1, chosen.reshape(-1, 1))
        apart = max(apart, (taken[:, 0] - seen.reshape(-1)).abs().max().item())
        advantage = ((reward - reward.mean()) / (reward.std() + 1e-6)).reshape(-1, 1)
        d = logp.exp() * advantage
        d.scatter_add_(1, chosen.reshape(-1, 1), -advantage)
        d = train.backward(d.div_(SEQUENCES * LENGTH), logits=raw)
        h = trainer.views[0][before.long()]
        torch.matmul(d.float().t(), h.float(), out=trainer.grads[1])
        trainer.grads[0].zero_().index_add_(0, before.long(), d.float() @ trainer.views[1].float())

        # the step, and its patch to the sampler
        _, clip = trainer.adam.grad_norm(1.0)
        trainer.adam.step(iteration, lr, grad_scale=clip, seed=seed)
        sampler.apply(trainer.encode())
        for served, view in zip(sampler.weights, trainer.views):
            if not torch.equal(served.view(torch.int16), view.view(torch.int16)):
                raise RuntimeError("the served weights differ from the trainer's view")
    return rewards, apart


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--iterations", type=int, default=30)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    rewards, apart = run(a.iterations, a.state_bits)
    print("mean reward:", " ".join(f"{r:.3f}" for r in rewards))
    print(f"log-probabilities of sampler and trainer differ by at most {apart:.2g}")


if __name__ == "__main__":
    main()
