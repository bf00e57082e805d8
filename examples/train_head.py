"""Trains the output layer of a small language model with the losses over rows
of logits, on synthetic data: first it learns from the largest logits of a
teacher, then sampled tokens with a reward move it by the clipped policy loss,
then ranked pairs of sequences by the preference loss.

    python examples/train_head.py [--steps 20]

Every loss writes the gradient of its logits in the same call; the layer's
own gradient is one matrix product from there.  The log-probabilities that the
later losses start from (the policy that sampled, the reference) come from the
library too, and so does their gradient in the last, plain step."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp32_reductions_amd as red  # noqa: E402

TOKENS, WIDTH, VOCABULARY, KEPT = 512, 64, 5003, 16


class Head:
    """logits = hidden @ weight in bf16, trained by plain gradient steps."""

    def __init__(self, generator, rate):
        self.weight = torch.randn(WIDTH, VOCABULARY, device="cuda", generator=generator) * 0.05
        self.rate = rate

    def logits(self, hidden):
        return (hidden @ self.weight).to(torch.bfloat16)

    def step(self, hidden, dlogits):
        self.weight -= self.rate * (hidden.t() @ dlogits.float())


def log_probabilities(logits, targets):
    """(ln p of the targets, log-sum-exp, entropy) of every row."""
    out = [torch.empty(len(targets), device="cuda") for _ in range(3)]
    red.token_logprob_bf16(logits, targets, out[0], out[1], entropy=out[2])
    return out


def distill(head, hidden, teacher, steps):
    """Divergence from the teacher's KEPT largest logits and the rest."""
    val, idx = teacher.topk(KEPT, dim=1)
    rest = teacher.logsumexp(1)
    loss, losses = torch.empty(1, device="cuda"), []
    for _ in range(steps):
        logits = head.logits(hidden)
        dlogits = torch.empty_like(logits)
        red.distill_topk_bf16(logits, idx, val, loss, dlogits=dlogits, teacher_lse=rest)
        head.step(hidden, dlogits)
        losses.append(loss.item())
    return losses


def improve(head, hidden, generator, steps):
    """Tokens sampled from the head, rewarded where they are even numbers."""
    logits = head.logits(hidden)
    tokens = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=generator).squeeze(1)
    old, _, _ = log_probabilities(logits, tokens)
    reward = (tokens % 2 == 0).float()
    advantage = (reward - reward.mean()) / (reward.std() + 1e-6)
    counted = torch.ones(len(tokens), device="cuda")
    counted[:64] = 0.0  # a prompt
    weight = counted / counted.sum()
    loss, logp, losses = torch.empty(1, device="cuda"), torch.empty_like(old), []
    for _ in range(steps):
        logits = head.logits(hidden)
        dlogits = torch.empty_like(logits)
        red.policy_loss_bf16(logits, tokens, old, advantage, loss, logp, dlogits=dlogits,
                             ref_logp=old, weight=weight, kl_coef=0.02, clip_high=0.28)
        head.step(hidden, dlogits)
        losses.append(loss.item())
    return losses


def prefer(head, hidden, generator, steps):
    """Eight packed sequences: the first four are preferred to the others."""
    tokens = torch.randint(VOCABULARY, (TOKENS,), device="cuda", generator=generator)
    starts = torch.tensor([0, 40, 128, 200, 256, 300, 380, 420, TOKENS], device="cuda")
    logp, _, _ = log_probabilities(head.logits(hidden), tokens)
    ref = torch.stack([logp[a:b].sum() for a, b in zip(starts[:-1].tolist(), starts[1:].tolist())])
    loss, seq, losses = torch.empty(1, device="cuda"), torch.empty_like(ref), []
    for _ in range(steps):
        logits = head.logits(hidden)
        dlogits = torch.empty_like(logits)
        red.preference_loss_bf16(logits, tokens, starts, loss, seq, dlogits=dlogits, ref_logp=ref,
                                 beta=0.1)
        head.step(hidden, dlogits)
        losses.append(loss.item())
    return losses


def imitate(head, hidden, generator, steps):
    """Plain maximum likelihood with an entropy bonus: both gradients in one
    call."""
    tokens = torch.randint(VOCABULARY, (TOKENS,), device="cuda", generator=generator)
    each = torch.full((TOKENS,), -1.0 / TOKENS, device="cuda")  # of the loss to ln p
    losses = []
    for _ in range(steps):
        logits = head.logits(hidden)
        logp, lse, entropy = log_probabilities(logits, tokens)
        red.token_logprob_grad_bf16(logits, tokens, lse, each, logits, entropy=entropy,
                                    gentropy=0.01 * each)
        head.step(hidden, logits)
        losses.append(-logp.mean().item())
    return losses


def main(steps=20):
    generator = torch.Generator(device="cuda").manual_seed(0)
    head = Head(generator, 1.0)
    hidden = torch.randn(TOKENS, WIDTH, device="cuda", generator=generator)
    teacher = hidden @ (torch.randn(WIDTH, VOCABULARY, device="cuda", generator=generator) * 0.3)
    history = {"distillation": distill(head, hidden, teacher, steps),
               "policy": improve(head, hidden, generator, steps),
               "preference": prefer(head, hidden, generator, steps),
               "likelihood": imitate(head, hidden, generator, steps)}
    for name, losses in history.items():
        print("%-13s %8.4f -> %8.4f" % (name, losses[0], losses[-1]))
    return history


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=20)
    main(parser.parse_args().steps)
