"""Distillation where the teacher or the student is far from ordinary: a
student whose listed logits lead all others so far that no other term is left
beside them, and the columns not listed without any probability; teachers with
NaN among their entries."""
import math

import pytest

import rowloss_reference as ref
from gpu_helpers import say
from test_gpu_rowloss import DTYPES, draw, f32, run_distill

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# Columns: a row held by a wave, by a workgroup, and one longer than that.
COLUMNS = [9, 1200, 6000, 150000]


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


def lists(n, V, K, g):
    return torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(n)])


def teacher_with_rest(val, scale, rest):
    """The log-sum-exp of a teacher whose entries leave `rest` to the others."""
    return ((val.double() * scale).logsumexp(1) - torch.log1p(-rest.double())).float()


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", COLUMNS)
def test_listed_logits_far_above_the_rest(red, V, t):
    """Every term outside the list is below 2^-126 of the row's largest; the
    rest's loss and gradient are those among the columns outside."""
    say("leading list V=%d %s" % (V, t))
    n, K = 7, 4
    g, z, _ = draw(n, V, t, V + 1, std=1.0)
    idx = lists(n, V, K, g)
    idx[4, 2] = -1
    for r, lead in enumerate((100.0, 150.0, 600.0, 90.0, 200.0, 120.0)):
        z[r, idx[r, 0]] = lead
    z[2, idx[2, 1:3]] = 599.0
    z[5, V // 2:] -= 150.0
    z[5, idx[5, 0]] = 120.0
    val = torch.randn(n, K, generator=g)
    rest = torch.tensor([0.1, 0.5, 1e-3, 0.9, 0.25, 0.1, 0.3])
    listed = torch.where(idx >= 0, val, torch.full_like(val, -math.inf))
    w = torch.rand(n, generator=g) + 0.5
    for scale in (1.0, 0.9):
        lse = teacher_with_rest(listed, scale, rest)
        run_distill(red, z, idx, val, t, scale, w, lse)
        run_distill(red, z, idx, val, t, scale, w, lse, grad=False)
        run_distill(red, z, idx, val, t, scale, w, lse, shift=1, pad=3, in_place=True)


def compact(z, idx):
    """The listed columns of every row alone, with entry k in column k."""
    return z.gather(1, idx), torch.arange(idx.shape[1]).repeat(z.shape[0], 1)


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", COLUMNS)
@pytest.mark.parametrize("lowest", [False, True])
def test_rounding_of_a_rest_without_columns(red, V, t, lowest):
    """The teacher lists every column that the student's mask leaves.  1 - Q is
    then what rounding left of the teacher's log-sum-exp, and no rest."""
    say("no columns outside V=%d %s %s" % (V, t, lowest))
    n, K = 24, 5
    mask = torch.finfo(DTYPES[t]).min if lowest else -math.inf
    g, z, _ = draw(n, V, t, V + 2)
    idx = lists(n, V, K, g)
    keep = torch.zeros(n, V, dtype=torch.bool).scatter_(1, idx, True)
    z[~keep] = mask
    val = torch.randn(n, K, generator=g) * 3 + 9.0
    lse = val.double().logsumexp(1).float()
    missing = 1 - (val.double() - lse.double().unsqueeze(1)).exp().sum(1)
    assert (missing > 0).sum() > 3 and (missing < 0).sum() > 3
    w = torch.rand(n, generator=g) + 0.5
    loss, row_loss, dz = f32(1), f32(n), torch.full_like(z, 7.0).cuda()
    getattr(red, "distill_topk_" + t)(z.cuda(), idx.cuda(), val.cuda(), loss, dlogits=dz,
                                      teacher_lse=lse.cuda(), weight=w.cuda(), row_loss=row_loss)
    few, at = compact(z, idx)
    want = ref.distill_topk(few, at, val, 1.0, w, lse)  # every column listed: no rest
    ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
    ref.check("row_loss", row_loss, *want["row_loss"])
    ref.check("dlogits", dz.cpu().gather(1, idx), *want["dlogits"])
    assert not dz.cpu()[~keep].any()


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", COLUMNS)
def test_a_real_rest_without_columns(red, V, t):
    """A rest that is more than rounding: infinite where the student has
    masked the columns outside, and -ln p_r of it where it has them lowest."""
    say("a rest of masked columns V=%d %s" % (V, t))
    low = torch.finfo(DTYPES[t]).min
    n, K = 4, 3
    g, z, _ = draw(n, V, t, V + 3)
    idx = lists(n, V, K, g)
    keep = torch.zeros(n, V, dtype=torch.bool).scatter_(1, idx, True)
    z[:2][~keep[:2]] = -math.inf
    z[2:3][~keep[2:3]] = low
    val = torch.randn(n, K, generator=g)
    rest = torch.tensor([0.25, 1e-4, 0.25, 0.25])
    lse = teacher_with_rest(val, 1.0, rest)
    w = torch.ones(n)
    loss, row_loss, dz = f32(1), f32(n), torch.full_like(z, 7.0).cuda()
    getattr(red, "distill_topk_" + t)(z.cuda(), idx.cuda(), val.cuda(), loss, dlogits=dz,
                                      teacher_lse=lse.cuda(), weight=w.cuda(), row_loss=row_loss)
    want = ref.distill_topk(z, idx, val, 1.0, w, lse)
    assert (want["row_loss"][0][:2] == math.inf).all() and loss.item() == math.inf
    ref.check("row_loss", row_loss, *want["row_loss"])
    some = torch.tensor([0, 1, 3])
    ref.check("dlogits", dz.cpu()[some], want["dlogits"][0][some], want["dlogits"][1][some])
    # Equal logits outside share the rest's gradient.  The sum of V equal terms
    # and its reciprocal, and the rounding of the result.
    d = dz.cpu()[2].double()
    q = (val[2].double() - lse[2].double()).exp()
    share = -(1 - q.sum()) / (V - K)
    bound = share.abs() * ref.stat_error(V) + ref.round_bound(share, z.dtype)
    assert (d[~keep[2]] - share).abs().max() <= bound
    ref.check("listed", d[idx[2]], want["dlogits"][0][2][idx[2]], want["dlogits"][1][2][idx[2]])


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", COLUMNS)
@pytest.mark.parametrize("tail", [False, True])
def test_nan_among_the_teachers_entries(red, V, t, tail):
    """A teacher that gives NaN makes NaN of its own row, however many of its
    entries are NaN; padding is not looked at, and entries of -inf alone are
    no teacher."""
    say("NaN teachers V=%d %s tail=%s" % (V, t, tail))
    n, K = 7, 4
    g, z, _ = draw(n, V, t, V + 4)
    idx = lists(n, V, K, g)
    val = torch.randn(n, K, generator=g)
    val[0, :] = math.nan
    val[1, 2] = math.nan
    val[2, :2], val[2, 2:] = math.nan, -math.inf
    val[3, :] = -math.inf
    val[4, 1], idx[4, 1] = math.nan, -1
    val[5, :], idx[5, :] = math.nan, -1
    lse = torch.full((n,), 2.5) if tail else None
    w = torch.rand(n, generator=g) + 0.5
    w[6] = 0.0
    val[6, :] = math.nan
    bad = torch.tensor([1, 1, 1, 0, 0, 0, 0], dtype=torch.bool)
    _, row_loss, dz = run_distill(red, z, idx, val, t, 1.0, w, lse)
    assert torch.equal(row_loss.cpu().isnan(), bad)
    assert dz.cpu()[bad].isnan().all() and not dz.cpu()[~bad].isnan().any()
    # and without those rows the loss is a number
    loss, _, _ = run_distill(red, z, idx, val, t, 1.0, torch.where(bad, 0.0, w), lse)
    assert loss.isfinite().all()


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", COLUMNS + [196088])
def test_small_row_losses_with_a_rest(red, V, t):
    """A student close to its teacher: row losses that are small differences of
    large terms.  In the row loss, with S = S_out + S_in,

        (Q + q_r) ln S - q_r ln S_out + (terms of exact logits),

    Q + q_r = 1, so an error d of S_out makes d (p_r - q_r) of it and an error e
    of S_in makes e p_in, p_in the student's listed probability.  d: the row's
    sum and its move to the row's maximum; e: the exponents, of at most 40, and
    K additions.  The loss itself is rounded once."""
    say("small row losses V=%d %s" % (V, t))
    n, K = 12, 8 if V > 9 else 3
    g, z, _ = draw(n, V, t, V + 6, std=2.0)
    idx = lists(n, V, K, g)
    p = torch.softmax(z.double(), 1)
    p_in = p.gather(1, idx).sum(1)
    # a teacher that has the list 1 % more or less likely
    val = z.gather(1, idx).float()
    lse = (z.double().logsumexp(1) + 0.01 * torch.randn(n, generator=g).double()).float()
    loss, row_loss = f32(1), f32(n)
    getattr(red, "distill_topk_" + t)(z.cuda(), idx.cuda(), val.cuda(), loss, teacher_lse=lse.cuda(),
                                      row_loss=row_loss)
    lnq = val.double() - lse.double().unsqueeze(1)
    q_r = 1 - lnq.exp().sum(1)
    out = torch.ones(n, V, dtype=torch.bool).scatter_(1, idx, False)
    p_r = (p * out).sum(1)
    lnp = torch.log_softmax(z.double(), 1).gather(1, idx)
    want = (lnq.exp() * (lnq - lnp)).sum(1) + q_r * (q_r.log() - p_r.log())
    moved = ref.U * (2 * 40 + 2)
    bound = ((ref.stat_error(V) + moved) * (p_r - q_r).abs() + (moved + K * ref.U) * p_in
             + want.abs() * ref.U + 2.0 ** -46)
    ref.check("row_loss", row_loss, want, bound)
