"""Losses over more rows than one launch covers: the row losses of all its
launches are one sum, rounded once."""
import math

import pytest

import rowloss_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PART = 1 << 20  # rows of one launch


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


def cancelling(rows, seed):
    """Factors whose first PART add up to some 800000, and the others to what
    takes that away but for a small remainder."""
    g = torch.Generator().manual_seed(seed)
    v = torch.rand(rows, generator=g) * 0.5 + 0.5
    more = rows - PART
    v[PART:] = (-v[:PART].double().sum() / more).float()
    v[PART] += 1.0
    return v


@pytest.mark.parametrize("old", [None, 3.0])
@pytest.mark.parametrize("rows", [PART + 5, PART + 40000, 2 * PART + 100])
def test_a_loss_of_several_launches_is_rounded_once(red, rows, old):
    """All rows are alike but for their factor, so the loss is the factors'
    sum times one row's loss.  fp64 sums are off by 2^-53 of the terms' sizes
    in each of at most rows / 4096 + 24 steps, and the result by half an fp32
    step."""
    say("%d rows, old loss %s" % (rows, old))
    V = 3
    v = cancelling(rows, rows)
    size, steps = v.double().abs().sum(), rows / 4096 + 24
    start = 0.0 if old is None else old
    z = torch.zeros(rows, V, device="cuda")
    y = torch.ones(rows, dtype=torch.long, device="cuda")

    def check(loss, one):
        want = start + v.double().sum() * one
        bound = want.abs() * ref.U + size * abs(one) * steps * 2.0 ** -53
        assert abs(loss.double().item() - want) <= bound, (loss.item(), want.item(), float(bound))

    # policy: logp = -ln 3 and old_logp its rounding, inside the clip's bounds
    logp = torch.empty(rows, device="cuda")
    log3 = torch.full((rows,), -math.log(3.0), device="cuda")
    loss = torch.full((1,), start, device="cuda")
    red.policy_loss_f32(z, y, log3, v.cuda(), loss, logp, weight=torch.ones(rows, device="cuda"),
                        accum=old is not None)
    check(loss, -math.exp(-math.log(3.0) - float(torch.tensor(-math.log(3.0)))))
    # distillation from one entry: ln 3 a row, weighted by the factors
    loss = torch.full((1,), start, device="cuda")
    red.distill_topk_f32(z, y.unsqueeze(1), torch.zeros(rows, 1, device="cuda"), loss,
                         weight=v.cuda(), accum=old is not None)
    check(loss, math.log(3.0))
