"""Many rows longer than the registers of a workgroup: the policy loss and the
distillation in chunks, of which all but one are read a second time."""
import pytest

import rowloss_reference as ref
from gpu_helpers import say
from test_gpu_rowloss import DTYPES, draw, f32, place, untouched

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# (rows, vectors of 16 bytes): more rows than are cut into segments, one vector
# past a workgroup's registers, a usual remainder, a third chunk, and rows on
# both sides of the number of compute units.
LONG = [(260, 16385), (130, 18992), (131, 32769)]


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


def rows_of(rows, vecs, t):
    V = vecs * (4 if t == "f32" else 8) + 3
    g, z, y = draw(rows, V, t, vecs)
    some = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1])
    # targets in the first chunk, the last one and outside the vectors
    y[0], y[1], y[rows // 2], y[rows - 2] = 5, V - 1, V - 40, V // 2
    w = torch.rand(rows, generator=g) + 0.1
    w[2], y[3] = 0.0, -100
    return g, z, y, w, some


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows,vecs", LONG)
@pytest.mark.parametrize("ent", [0.0, 0.1])
@pytest.mark.parametrize("in_place", [False, True])
def test_policy(red, rows, vecs, t, ent, in_place):
    say("policy %d rows of %d vectors %s ent=%g in place=%s" % (rows, vecs, t, ent, in_place))
    g, z, y, w, some = rows_of(rows, vecs, t)
    V = z.shape[1]
    adv = torch.randn(rows, generator=g)
    shift, pad = (3, 2) if in_place else (0, 5)
    zd, flat = place(z, shift, pad, 5.0)
    logp, lse = f32(rows), f32(rows)
    getattr(red, "token_logprob_" + t)(zd, y.cuda(), logp, lse)
    want = ref.token_logprob(z[some], y[some], 1.0)
    ref.check("logp", logp.cpu()[some], *want["logp"])
    old, rlogp = logp.cpu() + 0.05, logp.cpu() - 0.3
    dz = zd
    if not in_place:
        dz, flat = place(torch.full_like(z, 7.0), shift, pad, 5.0)
    loss, lp = f32(1), f32(rows)
    H = f32(rows) if ent else None
    getattr(red, "policy_loss_" + t)(zd, y.cuda(), old.cuda(), adv.cuda(), loss, lp, dlogits=dz,
                                     ref_logp=rlogp.cuda(), weight=w.cuda(), entropy=H,
                                     kl_coef=0.1, entropy_coef=ent)
    want = ref.policy_loss(z[some], y[some], old[some], adv[some], w[some], 1.0, rlogp[some],
                           kl_coef=0.1, entropy_coef=ent)
    ref.check("logp", lp.cpu()[some], *want["logp"])
    if ent:
        ref.check("entropy", H.cpu()[some], *want["entropy"])
    ref.check("dlogits", dz.cpu()[some], *want["dlogits"])
    assert loss.isfinite().all() and not dz[2:4].any() and not lp[2:4].any()
    assert untouched(flat, shift, rows, V, pad, 5.0)


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows,vecs", LONG)
@pytest.mark.parametrize("tail", [False, True])
def test_distill(red, rows, vecs, t, tail):
    say("distill %d rows of %d vectors %s tail=%s" % (rows, vecs, t, tail))
    g, z, _, w, some = rows_of(rows, vecs, t)
    V = z.shape[1]
    idx = torch.randint(V // 9, (rows, 9), generator=g) + torch.arange(9) * (V // 9)
    idx[:, 8] = V - 1
    val = torch.randn(rows, 9, generator=g) * 2
    lse = val.double().logsumexp(1).float() + 0.4 if tail else None
    for in_place in (False, True):
        zd, flat = place(z, 1, 4, 5.0)
        dz = zd
        if not in_place:
            dz, flat = place(torch.full_like(z, 7.0), 1, 4, 5.0)
        loss, row_loss = f32(1), f32(rows)
        getattr(red, "distill_topk_" + t)(zd, idx.cuda(), val.cuda(), loss, dlogits=dz,
                                          teacher_lse=None if lse is None else lse.cuda(),
                                          weight=w.cuda(), row_loss=row_loss)
        want = ref.distill_topk(z[some], idx[some], val[some], 1.0, w[some],
                                None if lse is None else lse[some])
        ref.check("row_loss", row_loss.cpu()[some], *want["row_loss"])
        ref.check("dlogits", dz.cpu()[some], *want["dlogits"])
        assert loss.isfinite().all() and not dz[2].any()
        assert untouched(flat, 1, rows, V, 4, 5.0)
