"""The losses over rows of logits by the number of rows: on both sides of
every count that changes how rows are shared out (a row's threads, segments of
few long rows, groups of arrivals at the loss, pairs with and without a kernel
of their own), and one call after another on one workspace."""
import math

import pytest

import rowloss_reference as ref
from gpu_helpers import say
from test_gpu_rowloss import (DTYPES, draw, f32, place, policy_inputs, run_distill, run_grad,
                              run_logprob, run_policy, run_preference, teacher)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


def check_rows(name, got, want, rows):
    """got[rows] against the reference of those rows alone."""
    ref.check(name, got.cpu()[rows], *want)


# Columns for every number of threads and vectors that a row is given where
# rows are more than compute units, and where they are not.
MANY = [(300, 500), (300, 2040), (300, 4090), (300, 8170), (261, 16380), (261, 33000),
        (258, 65600), (257, 131072), (100, 900), (256, 4100), (200, 30001), (140, 65540)]


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows,V", MANY)
def test_many_rows(red, rows, V, t):
    say("%d rows of %d %s" % (rows, V, t))
    V = V // 2 if t == "f32" else V
    g, z, y = draw(rows, V, t, V)
    some = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1])
    w = torch.rand(rows, generator=g) + 0.1
    dead = torch.rand(rows, generator=g) < 0.2
    dead[some] = False
    w[dead] = 0.0
    zd, _ = place(z)
    # policy, with the entropy and without
    stat = {"logp": f32(rows), "lse": f32(rows)}
    getattr(red, "token_logprob_" + t)(zd, y.cuda(), stat["logp"], stat["lse"])
    want = ref.token_logprob(z[some], y[some], 1.0)
    check_rows("logp", stat["logp"], want["logp"], some)
    check_rows("lse", stat["lse"], want["lse"], some)
    logp = stat["logp"].cpu()
    adv = torch.randn(rows, generator=g)
    old, rlogp = logp + 0.05, logp - 0.3
    for ent in (0.0, 0.1):
        loss, lp, dz = f32(1), f32(rows), torch.full_like(z, 7.0).cuda()
        getattr(red, "policy_loss_" + t)(zd, y.cuda(), old.cuda(), adv.cuda(), loss, lp,
                                         dlogits=dz, ref_logp=rlogp.cuda(), weight=w.cuda(),
                                         kl_coef=0.1, entropy_coef=ent)
        want = ref.policy_loss(z[some], y[some], old[some], adv[some], w[some], 1.0, rlogp[some],
                               kl_coef=0.1, entropy_coef=ent)
        check_rows("logp", lp, want["logp"], some)
        check_rows("dlogits", dz, want["dlogits"], some)
        assert not dz.cpu()[dead].any() and not lp.cpu()[dead].any()
        if not ent:
            # the loss from the rows' own log-probabilities, each off by half a step
            x = lp.cpu().double()
            ratio = (x - old.double()).exp()
            d = rlogp.double() - x
            clip = float(torch.tensor(0.2))
            row = -torch.minimum(ratio * adv.double(),
                                 ratio.clamp(1 - clip, 1 + clip) * adv.double())
            kl = float(torch.tensor(0.1))
            row = row + kl * (torch.expm1(d) - d)
            off = (ratio * adv.double()).abs() + kl * torch.expm1(d).abs()
            wd = w.double()
            bound = (wd * off * (x.abs() * ref.U * 1.01)).sum()
            total = (wd * row)[~dead].sum()
            assert abs(loss.item() - total) <= bound + abs(total) * 2 * ref.U
    # distillation, with the rest and without
    idx = torch.stack([torch.randperm(V, generator=g)[:7] for _ in range(rows)])
    val = torch.randn(rows, 7, generator=g) * 2
    for lse in (None, val.double().logsumexp(1).float() + 0.4):
        loss, row_loss, dz = f32(1), f32(rows), torch.full_like(z, 7.0).cuda()
        getattr(red, "distill_topk_" + t)(zd, idx.cuda(), val.cuda(), loss, dlogits=dz,
                                          teacher_lse=None if lse is None else lse.cuda(),
                                          weight=w.cuda(), row_loss=row_loss)
        want = ref.distill_topk(z[some], idx[some], val[some], 1.0, w[some],
                                None if lse is None else lse[some])
        check_rows("row_loss", row_loss, want["row_loss"], some)
        check_rows("dlogits", dz, want["dlogits"], some)
        assert not dz.cpu()[dead].any()
        rl = row_loss.cpu().double() * w.double()
        assert abs(loss.item() - rl.sum()) <= (rl.abs().sum() + abs(rl.sum())) * ref.U * 1.01


@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 127, 128, 129, 191, 1000, 4095, 4097, 16383,
                                  16384, 16385, 20000])
def test_rows_that_join(red, rows):
    """Every row counts once in the sum, whatever group it arrives in."""
    say("%d rows join" % rows)
    _, z, y = draw(rows, 24, "bf16", rows)
    for k in range(2):  # the second call finds the counts as the first one left them
        run_policy(red, z, y, "bf16", rows + k)
        idx, val, lse = teacher(z, 3, k, k == 1, 1.0)
        run_distill(red, z, idx, val, "bf16", 1.0, None, lse, grad=k == 0)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("vecs", [6143, 6144, 6145, 8191, 8193, 16385])
@pytest.mark.parametrize("rows", [1, 5, 64, 65])
def test_few_long_rows(red, rows, vecs, t):
    """Around the lengths and counts from which rows are cut into segments,
    with a target in every part of a row."""
    V = vecs * (4 if t == "f32" else 8) + 3
    say("%d rows of %d %s" % (rows, V, t))
    rows = min(rows, 5) if vecs > 8193 and rows < 64 else rows
    g, z, y = draw(rows, V, t, V)
    y[0] = V - 1
    if rows > 4:
        y[1], y[2], y[3] = 0, V // 2, -100
        z[4, V // 3:] = -math.inf  # whole segments without a finite logit
        y[4] = 5
    run_logprob(red, z, y, t, 1.0)
    if rows <= 5:
        run_logprob(red, z, y, t, 0.7, shift=1, pad=2)
        run_policy(red, z, y, t, 1, ent=0.1, entropy_out=True)
        run_policy(red, z, y, t, 2, shift=1, pad=2, in_place=True)
        run_preference(red, z, y, t, torch.tensor([0, rows // 2, rows]))
    else:
        run_policy(red, z, y, t, 1)


def test_hundred_long_rows(red):
    for rows in (128, 129):
        _, z, y = draw(rows, 65544, "bf16", rows)
        run_logprob(red, z, y, "bf16", 1.0)


@pytest.mark.parametrize("rows", [90, 256, 257, 600])
@pytest.mark.parametrize("pairs", [1, 2, 30, 31, 32, 64])
def test_numbers_of_pairs(red, rows, pairs):
    """Ragged sequences, some empty, some rows in none, with both ways to
    finish a pair; targets that do not count."""
    say("%d pairs, %d rows" % (pairs, rows))
    g, z, y = draw(rows, 77, "bf16", rows + pairs)
    y[torch.rand(rows, generator=g) < 0.1] = -1
    starts = torch.randint(rows + 1, (2 * pairs + 1,), generator=g).sort().values
    starts[pairs // 2 + 1] = starts[pairs // 2]  # an empty sequence
    refs = torch.randn(2 * pairs, generator=g)
    w = torch.rand(pairs, generator=g)
    for average in (False, True):
        run_preference(red, z, y, "bf16", starts.sort().values, w, refs, average=average,
                       beta=0.02)
    run_preference(red, z, y, "bf16", torch.full((2 * pairs + 1,), rows // 3), w, refs)  # nothing


def test_falling_starts_leave_the_workspace_sound(red):
    """Starts have to be nondecreasing; where they are not, the results mean
    nothing, and the next call is right."""
    g, z, y = draw(100, 50, "bf16", 1)
    loss, seq = f32(1), f32(6)
    for starts in ([50, 20, 80, 10, 100, 0, 70], [90, -4, 300, 2, 2, 1, 0]):
        red.preference_loss_bf16(z.cuda(), y.cuda(), torch.tensor(starts).cuda(), loss, seq)
        run_preference(red, z, y, "bf16", torch.tensor([0, 20, 50, 60, 80, 90, 100]))


def test_gradient_of_many_rows(red):
    for rows, V in ((700, 300), (300, 5000)):
        _, z, y = draw(rows, V, "bf16", V)
        run_grad(red, z, y, "bf16", 1.0, 1, True)


def test_calls_of_every_kind_share_a_workspace(red):
    """Split rows, joined rows, joined pairs and the library's other
    reductions in turn: the counts and partial results of one are no
    other's."""
    _, long_z, long_y = draw(3, 70001, "f32", 1)
    _, z, y = draw(150, 600, "bf16", 2)
    x = torch.rand(1 << 20, device="cuda")
    out = torch.zeros(1, device="cuda")
    total = x.double().sum().item()
    for k in range(3):
        run_policy(red, long_z, long_y, "f32", k)
        run_policy(red, z, y, "bf16", k)
        red.sum_f32(x, out)
        assert abs(out.item() - total) <= total * 1e-6
        run_preference(red, z, y, "bf16", torch.tensor([0, 40, 70, 100, 150]))
        idx, val, lse = teacher(z, 9, k, True, 1.0)
        run_distill(red, z, idx, val, "bf16", 1.0, None, lse)
        run_logprob(red, long_z, long_y, "f32", 1.0)


@pytest.mark.parametrize("cus", ["8", "304"])
def test_other_device_sizes(red, monkeypatch, cus):
    """The plans of other numbers of compute units give the same losses."""
    monkeypatch.setenv("RED_TEST_CUS", cus)
    for rows, V in ((40, 3000), (12, 40000), (270, 900)):
        _, z, y = draw(rows, V, "bf16", V)
        run_policy(red, z, y, "bf16", 1, ent=0.1)
        run_logprob(red, z, y, "bf16", 1.0)
        run_preference(red, z, y, "bf16", torch.tensor([0, rows // 3, rows]))
        idx, val, lse = teacher(z, 9, 1, True, 1.0)
        run_distill(red, z, idx, val, "bf16", 1.0, None, lse)
