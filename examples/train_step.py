"""The end of a language model's training step on synthetic data: a residual stream
goes through the final norm, a router that chooses experts for its rows is kept in
balance, and the rows meet a large output layer whose logits are never stored.

    python examples/train_step.py [--steps 10]

Both losses add up in one value on the GPU, and each call that takes part in it
writes its gradients with it; the norm's gradient joins them.  The layer and the
router take plain gradient steps."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp32_reductions_amd as red  # noqa: E402

TOKENS, WIDTH, VOCABULARY, EXPERTS, CHOSEN = 512, 256, 20011, 16, 2
BALANCE, Z_ROUTER, Z_HEAD = 0.01, 0.001, 1e-4


class Step:
    """Weights, and the buffers that every step uses again."""

    def __init__(self, generator):
        def normal(*shape, std):
            return (torch.randn(*shape, device="cuda", generator=generator) * std).bfloat16()

        self.norm = normal(WIDTH, std=0.1) + 1.0
        self.layer = normal(VOCABULARY, WIDTH, std=0.05)
        self.router = normal(EXPERTS, WIDTH, std=0.05)
        self.loss = torch.zeros(1, device="cuda")
        self.counts = torch.zeros(EXPERTS, dtype=torch.int64, device="cuda")
        self.rstd, self.logp = (torch.empty(TOKENS, device="cuda") for _ in range(2))

    def losses(self, x, residual, targets, weight):
        """The loss and every gradient: (of x and the residual, the norm's weight, the
        output layer, the router)."""
        h, y, dy, dx = (torch.empty_like(x) for _ in range(4))
        red.add_rmsnorm_bf16(x, self.norm, y, residual=residual, sum=h, rstd=self.rstd)

        dlayer = torch.empty_like(self.layer)
        red.linear_ce_bf16(y, self.layer, targets, self.loss, logp=self.logp, dhidden=dy,
                           dweight=dlayer, row_weight=weight, z_coef=Z_HEAD)

        logits = y @ self.router.t()
        experts = logits.topk(CHOSEN, dim=1).indices
        dlogits = torch.empty_like(logits)
        red.router_balance_bf16(logits, experts, self.loss, self.counts, dlogits=dlogits,
                                weight=weight, balance_coef=BALANCE, z_coef=Z_ROUTER, accum=True)
        drouter = dlogits.t() @ y
        dy += dlogits @ self.router

        dnorm = torch.empty(WIDTH, device="cuda")
        red.rmsnorm_grad_bf16(h, self.norm, self.rstd, dy, dx, dweight=dnorm)
        return dx, dnorm, dlayer, drouter

    def update(self, gradients, rate):
        _, dnorm, dlayer, drouter = gradients
        self.norm -= (rate * dnorm).bfloat16()
        self.layer -= rate * dlayer
        self.router -= rate * drouter


def batch(generator):
    """Rows of a block's output and of the residual stream, targets, and the weights
    of a batch whose first quarter is a prompt."""
    x = torch.randn(TOKENS, WIDTH, device="cuda", generator=generator).bfloat16()
    residual = (torch.randn(TOKENS, WIDTH, device="cuda", generator=generator) * 2).bfloat16()
    targets = torch.randint(VOCABULARY, (TOKENS,), device="cuda", generator=generator)
    counted = torch.ones(TOKENS, device="cuda")
    counted[:TOKENS // 4] = 0.0
    return x, residual, targets, counted / counted.sum()


def main(steps=10):
    generator = torch.Generator(device="cuda").manual_seed(0)
    step = Step(generator)
    data = batch(generator)
    losses = []
    for _ in range(steps):
        step.update(step.losses(*data), 0.5)
        losses.append(step.loss.item())
    print("loss %8.4f -> %8.4f, rows of the busiest expert %d of %d"
          % (losses[0], losses[-1], step.counts.max(), step.counts.sum()))
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=10)
    main(parser.parse_args().steps)
