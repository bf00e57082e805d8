"""The fp64 reference of the losses over rows of logits against central
differences and automatic differentiation of its own losses, and against a
few values known in closed form (no GPU needed)."""
import math

import pytest
import torch

import rowloss_reference as ref


def case(rows, V, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, V, generator=g, dtype=torch.double) * 2
    y = torch.randint(V, (rows,), generator=g)
    return g, z, y


def numeric(loss, z, step=1e-5):
    d = torch.zeros_like(z)
    for i in range(z.shape[0]):
        for j in range(z.shape[1]):
            e = torch.zeros_like(z)
            e[i, j] = step
            d[i, j] = (loss(z + e) - loss(z - e)) / (2 * step)
    return d


def close(a, b):
    assert torch.allclose(a, b, rtol=1e-6, atol=1e-8), (a - b).abs().max()


@pytest.mark.parametrize("entropy", [False, True])
def test_token_logprob_gradient(entropy):
    g, z, y = case(4, 7, 1)
    y[2] = -100
    scale = 0.5
    glogp, gent = torch.randn(2, 4, generator=g, dtype=torch.double)

    def loss(z):
        out = ref.token_logprob(z, y, scale)
        return (glogp * out["logp"][0]).sum() + entropy * (gent * out["entropy"][0]).sum()

    out = ref.token_logprob(z, y, scale)
    d, _ = ref.token_logprob_grad(z, y, scale, out["lse"][0], glogp,
                                  gent if entropy else None, out["entropy"][0])
    close(d, numeric(loss, z))


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient(tail):
    g, z, _ = case(5, 9, 2)
    idx = torch.stack([torch.randperm(9, generator=g)[:4] for _ in range(5)])
    idx[1, 2] = -1
    idx[2, 3] = idx[2, 0]
    t = torch.randn(5, 9, generator=g, dtype=torch.double)
    val = t.gather(1, idx.clamp_min(0)) - (math.log(2.0) if tail else 0.0)
    lse = (t * 0.5).logsumexp(1) if tail else None
    w = torch.tensor([0.3, 0.2, 0.1, 0.0, 0.4], dtype=torch.double)
    out = ref.distill_topk(z, idx, val, 0.5, w, lse)
    close(out["dlogits"][0],
          numeric(lambda z: ref.distill_topk(z, idx, val, 0.5, w, lse)["loss"][0], z))
    assert (out["row_loss"][0][torch.arange(5) != 2] >= -1e-12).all()


@pytest.mark.parametrize("kl,ent", [(0.0, 0.0), (0.1, 0.0), (0.05, 0.02)])
def test_policy_gradient(kl, ent):
    g, z, y = case(6, 8, 3)
    y[4] = 8
    logp = ref.token_logprob(z, y, 1.0)["logp"][0]
    old = logp - torch.tensor([0.0, 0.5, -0.5, 0.1, 0.0, 0.5], dtype=torch.double)
    adv = torch.tensor([1.0, 1.0, -1.0, -2.0, 1.0, -1.0], dtype=torch.double)
    w = torch.tensor([0.5, 0.25, 0.25, 1.0, 1.0, 0.0], dtype=torch.double)
    args = dict(ref_logp=logp + 0.3, kl_coef=kl, entropy_coef=ent)
    out = ref.policy_loss(z, y, old, adv, w, **args)
    close(out["dlogits"][0],
          numeric(lambda z: ref.policy_loss(z, y, old, adv, w, **args)["loss"][0], z))


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
def test_preference_gradient(kind, average):
    g, z, y = case(11, 6, 4)
    y[3] = -1
    starts = torch.tensor([0, 3, 5, 5, 9])
    w = torch.tensor([0.6, 0.4], dtype=torch.double)
    r = torch.randn(4, generator=g, dtype=torch.double)
    args = dict(ref_logp=r, kind=kind, beta=0.3, margin=0.2, smoothing=0.1, average=average)
    out = ref.preference_loss(z, y, starts, w, **args)
    close(out["dlogits"][0],
          numeric(lambda z: ref.preference_loss(z, y, starts, w, **args)["loss"][0], z))
    assert (out["dlogits"][0][9:] == 0).all()


def test_closed_forms():
    z = torch.full((1, 16), 3.0)
    out = ref.token_logprob(z, torch.tensor([5]), 1.0)
    assert abs(out["logp"][0].item() + math.log(16)) < 1e-14
    assert abs(out["entropy"][0].item() - math.log(16)) < 1e-14
    # a teacher equal to the student costs nothing
    g, z, _ = case(3, 10, 5)
    idx = torch.arange(10).repeat(3, 1)
    out = ref.distill_topk(z, idx, z, 1.0, torch.ones(3, dtype=torch.double))
    assert out["loss"][0].abs() < 1e-12 and out["dlogits"][0].abs().max() < 1e-12
    out = ref.distill_topk(z, idx[:, :4], z[:, :4], 1.0, torch.ones(3, dtype=torch.double),
                           z.logsumexp(1))
    assert out["loss"][0].abs() < 1e-12 and out["dlogits"][0].abs().max() < 1e-12
    # equal sequences: ln 2
    z = torch.zeros(4, 5, dtype=torch.double)
    out = ref.preference_loss(z, torch.zeros(4, dtype=torch.long), torch.tensor([0, 2, 4]),
                              torch.ones(1, dtype=torch.double))
    assert abs(out["loss"][0].item() - math.log(2)) < 1e-14
