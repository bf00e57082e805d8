"""The losses over rows of logits on the GPU against the fp64 reference
(rowloss_reference.py), whose bounds follow from the formats and the lengths.

Sizes sit on both sides of every boundary of the kernels: rows shorter than a
vector, around each number of threads and vectors a row is given, rows longer
than a workgroup's registers; bases that are aligned to their element only;
padded strides; masks that leave a row empty."""
import math

import pytest

import rowloss_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# (columns, rows)
SHAPES = [(1, 3), (2, 5), (3, 4), (7, 3), (8, 3), (9, 6), (15, 2), (17, 3), (64, 5), (127, 3),
          (500, 9), (1000, 6), (2047, 3), (2049, 3), (4096, 2), (4099, 3), (8191, 2), (8200, 2),
          (16384, 2), (16391, 3), (32768, 2), (32771, 2), (50001, 2), (65543, 2)]
LONG = [(131072, 1), (131081, 2), (262147, 1)]
CASES = [(v, r, t) for v, r in SHAPES for t in DTYPES] + [
    (v, r, t) for v, r in LONG for t in ("f32", "bf16")]


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


def draw(rows, V, dtype, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(rows, V, generator=g) * std).to(DTYPES[dtype])
    y = torch.randint(V, (rows,), generator=g)
    return g, z, y


def place(z, shift=0, pad=0, fill=math.nan):
    """z on the device, `shift` elements past a 256-byte boundary, rows `pad`
    elements apart; everything around it holds `fill`."""
    rows, V = z.shape
    flat = torch.full((shift + rows * (V + pad) + 8,), fill, dtype=z.dtype, device="cuda")
    view = flat[shift:shift + rows * (V + pad)].view(rows, V + pad)[:, :V]
    view.copy_(z)
    return view, flat


def untouched(flat, shift, rows, V, pad, fill):
    """Everything of `flat` but its rows still holds `fill`."""
    keep = torch.ones_like(flat, dtype=torch.bool)
    keep[shift:shift + rows * (V + pad)].view(rows, V + pad)[:, :V] = False
    rest = flat[keep]
    return bool((rest == fill).all()) if fill == fill else bool(rest.isnan().all())


def f32(n, fill=None):
    return torch.empty(n, device="cuda") if fill is None else torch.full((n,), fill, device="cuda")


def cuda(t):
    return None if t is None else t.cuda()


# --- one call of each operator, checked --------------------------------------

def run_logprob(red, z, y, t, scale, shift=0, pad=0, entropy=True):
    zd, _ = place(z, shift, pad)
    n = z.shape[0]
    out = {"logp": f32(n), "lse": f32(n), "entropy": f32(n) if entropy else None}
    getattr(red, "token_logprob_" + t)(zd, y.cuda(), out["logp"], out["lse"],
                                       entropy=out["entropy"], scale=scale)
    want = ref.token_logprob(z, y, scale)
    for k, v in out.items():
        if v is not None:
            ref.check(k, v, *want[k])
    return out


def gradient_buffer(z, shift, pad):
    return place(torch.full_like(z, 7.0), shift, pad, 5.0)


def run_grad(red, z, y, t, scale, seed, entropy, shift=0, pad=0, gshift=0, gpad=0):
    n, V = z.shape
    g = torch.Generator().manual_seed(seed)
    glogp = torch.randn(n, generator=g)
    gent = torch.randn(n, generator=g) if entropy else None
    stat = ref.token_logprob(z, y, scale)
    lse, H = stat["lse"][0].float(), stat["entropy"][0].float()
    zd, _ = place(z, shift, pad)
    dz, flat = gradient_buffer(z, gshift, gpad)
    getattr(red, "token_logprob_grad_" + t)(
        zd, y.cuda(), lse.cuda(), glogp.cuda(), dz, entropy=H.cuda() if entropy else None,
        gentropy=cuda(gent), scale=scale)
    ref.check("dlogits", dz, *ref.token_logprob_grad(z, y, scale, lse, glogp, gent, H))
    assert untouched(flat, gshift, n, V, gpad, 5.0)


def teacher(z, K, seed, tail, scale):
    n, V = z.shape
    g = torch.Generator().manual_seed(seed)
    t = z.float() + torch.randn(n, V, generator=g)
    val, idx = t.topk(min(K, V), dim=1)
    lse = (t.double() * scale).logsumexp(1).float() if tail else None
    return idx, val, lse


def run_distill(red, z, idx, val, t, scale, weight, lse, grad=True, shift=0, pad=0, gshift=0,
                gpad=0, in_place=False):
    n, V = z.shape
    zd, flat = place(z, shift, pad, 5.0 if in_place else math.nan)
    dz = None
    if in_place:
        dz, gshift, gpad = zd, shift, pad
    elif grad:
        dz, flat = gradient_buffer(z, gshift, gpad)
    loss, row_loss = f32(1, 0.25), f32(n)
    getattr(red, "distill_topk_" + t)(zd, idx.cuda(), val.cuda(), loss, dlogits=dz,
                                      teacher_lse=cuda(lse), weight=cuda(weight),
                                      row_loss=row_loss, scale=scale)
    w = weight if weight is not None else torch.full((n,), 1.0 / n)
    want = ref.distill_topk(z, idx, val, scale, w, lse)
    ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
    ref.check("row_loss", row_loss, *want["row_loss"])
    if dz is not None:
        ref.check("dlogits", dz, *want["dlogits"])
        assert untouched(flat, gshift, n, V, gpad, 5.0)
    return loss, row_loss, dz


def policy_inputs(z, y, seed, scale=1.0):
    n = z.shape[0]
    g = torch.Generator().manual_seed(seed)
    logp = ref.token_logprob(z, y, scale)["logp"][0].float()
    drift = torch.randn(n, generator=g) * 0.3
    for edge in (math.log(0.8), math.log(1.3)):  # no row on the kink
        drift = torch.where((drift - edge).abs() < 1e-2, edge + 1e-2, drift)
    return (logp - drift, torch.randn(n, generator=g), logp + torch.randn(n, generator=g) * 0.5,
            torch.rand(n, generator=g) / n)


def run_policy(red, z, y, t, seed, scale=1.0, ref_on=True, ent=0.0, weight="draw", grad=True,
               entropy_out=False, shift=0, pad=0, gshift=0, gpad=0, in_place=False):
    n, V = z.shape
    old, adv, rlogp, w = policy_inputs(z, y, seed, scale)
    w = w if isinstance(weight, str) else weight
    zd, flat = place(z, shift, pad, 5.0 if in_place else math.nan)
    dz = None
    if in_place:
        dz, gshift, gpad = zd, shift, pad
    elif grad:
        dz, flat = gradient_buffer(z, gshift, gpad)
    loss, logp = f32(1, 0.25), f32(n)
    H = f32(n) if entropy_out else None
    coef = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1 if ref_on else 0.0, entropy_coef=ent)
    getattr(red, "policy_loss_" + t)(zd, y.cuda(), old.cuda(), adv.cuda(), loss, logp, dlogits=dz,
                                     ref_logp=rlogp.cuda() if ref_on else None, weight=cuda(w),
                                     entropy=H, scale=scale, **coef)
    want = ref.policy_loss(z, y, old, adv, w if w is not None else torch.full((n,), 1.0 / n),
                           scale, rlogp, **coef)
    ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
    ref.check("logp", logp, *want["logp"])
    if entropy_out:
        ref.check("entropy", H, *want["entropy"])
    if dz is not None:
        ref.check("dlogits", dz, *want["dlogits"])
        assert untouched(flat, gshift, n, V, gpad, 5.0)
    return loss, logp, dz


def run_preference(red, z, y, t, starts, weight=None, ref_logp=None, grad=True, shift=0, pad=0,
                   gshift=0, gpad=0, in_place=False, **args):
    n, V = z.shape
    pairs = len(starts) // 2
    zd, flat = place(z, shift, pad, 5.0 if in_place else math.nan)
    dz = None
    if in_place:
        dz, gshift, gpad = zd, shift, pad
    elif grad:
        dz, flat = gradient_buffer(z, gshift, gpad)
    loss, seq = f32(1, 0.25), f32(2 * pairs)
    getattr(red, "preference_loss_" + t)(zd, y.cuda(), starts.cuda(), loss, seq, dlogits=dz,
                                         ref_logp=cuda(ref_logp), weight=cuda(weight), **args)
    w = weight if weight is not None else torch.full((pairs,), 1.0 / pairs, dtype=torch.double)
    want = ref.preference_loss(z, y, starts, w, ref_logp, **args)
    ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
    ref.check("seq_logp", seq, *want["seq_logp"])
    if dz is not None:
        ref.check("dlogits", dz, *want["dlogits"])
        assert untouched(flat, gshift, n, V, gpad, 5.0)
    return loss, seq, dz


# --- every length -------------------------------------------------------------

@pytest.mark.parametrize("V,rows,t", CASES)
def test_logprob(red, V, rows, t):
    say("token_logprob V=%d rows=%d %s" % (V, rows, t))
    _, z, y = draw(rows, V, t, V + rows)
    y[-1] = -100
    run_logprob(red, z, y, t, 1.0)
    run_logprob(red, z, y, t, 1 / 0.7, entropy=False)


@pytest.mark.parametrize("V,rows,t", CASES)
def test_logprob_grad(red, V, rows, t):
    say("token_logprob_grad V=%d rows=%d %s" % (V, rows, t))
    _, z, y = draw(rows, V, t, V + rows)
    y[-1] = V if rows > 1 else y[-1]
    run_grad(red, z, y, t, 1.0, 1, False)
    run_grad(red, z, y, t, 1 / 0.7, 2, True)


@pytest.mark.parametrize("V,rows,t", CASES)
def test_distill(red, V, rows, t):
    say("distill_topk V=%d rows=%d %s" % (V, rows, t))
    g, z, _ = draw(rows, V, t, V + rows)
    w = torch.rand(rows, generator=g)
    for tail in (False, True):
        idx, val, lse = teacher(z, 5 if V < 4000 else 70, V, tail, 0.5)
        run_distill(red, z, idx, val, t, 0.5, w, lse)
        run_distill(red, z, idx, val, t, 0.5, None, lse, grad=False)


@pytest.mark.parametrize("V,rows,t", CASES)
def test_policy(red, V, rows, t):
    say("policy_loss V=%d rows=%d %s" % (V, rows, t))
    _, z, y = draw(rows, V, t, V + rows)
    run_policy(red, z, y, t, 1)
    run_policy(red, z, y, t, 2, scale=1 / 0.8, ref_on=False, ent=0.05, entropy_out=True)
    run_policy(red, z, y, t, 3, ent=0.05, weight=None, grad=False)


@pytest.mark.parametrize("V,rows,t", CASES)
def test_preference(red, V, rows, t):
    rows += 3
    say("preference_loss V=%d rows=%d %s" % (V, rows, t))
    g, z, y = draw(rows, V, t, V + rows)
    starts = torch.tensor([0, rows // 2, rows])
    run_preference(red, z, y, t, starts)
    run_preference(red, z, y, t, starts, average=True, kind="squared", beta=0.5, grad=False)


# --- layouts --------------------------------------------------------------------

LAYOUTS = [(1, 0, 0, 0), (3, 5, 0, 0), (0, 0, 1, 3), (2, 1, 5, 2), (7, 9, 7, 9)]


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", [5, 501, 4101, 20001])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_strides_and_alignments(red, V, t, layout):
    say("layout %s V=%d %s" % (layout, V, t))
    shift, pad, gshift, gpad = layout
    where = dict(shift=shift, pad=pad, gshift=gshift, gpad=gpad)
    g, z, y = draw(5, V, t, V)
    run_logprob(red, z, y, t, 1.0, shift, pad)
    run_grad(red, z, y, t, 1.0, 3, True, **where)
    for tail in (False, True):
        idx, val, lse = teacher(z, 4, V, tail, 1.0)
        run_distill(red, z, idx, val, t, 1.0, None, lse, **where)
    run_policy(red, z, y, t, 4, ent=0.1, **where)
    run_preference(red, z, y, t, torch.tensor([0, 2, 5]), **where)


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", [3, 1001, 9000, 40003, 140001])
def test_gradient_over_its_logits(red, V, t):
    say("in place V=%d %s" % (V, t))
    g, z, y = draw(4, V, t, V + 1)
    for shift, pad in ((0, 0), (3, 2)):
        where = dict(shift=shift, pad=pad, in_place=True)
        run_policy(red, z, y, t, 5, ent=0.1, **where)
        for tail in (False, True):
            idx, val, lse = teacher(z, 6, V, tail, 1.0)
            run_distill(red, z, idx, val, t, 1.0, None, lse, **where)
        run_preference(red, z, y, t, torch.tensor([0, 2, 4]), **where)
        # the plain gradient, which has a call of its own
        stat = ref.token_logprob(z, y, 1.0)
        lse = stat["lse"][0].float()
        one = torch.ones(4)
        zd, flat = place(z, shift, pad, 5.0)
        getattr(red, "token_logprob_grad_" + t)(zd, y.cuda(), lse.cuda(), one.cuda(), zd)
        ref.check("dlogits", zd, *ref.token_logprob_grad(z, y, 1.0, lse, one))
        assert untouched(flat, shift, 4, V, pad, 5.0)


def test_offsets_past_32_bits(red):
    """The last rows of a matrix of more than 2^32 bytes and 2^31 elements."""
    V, rows = 65536, 33000
    say("policy_loss and token_logprob over %d x %d bf16" % (rows, V))
    z = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    _, tail, y = draw(3, V, "bf16", 9)
    z[-3:] = tail.cuda()
    targets = torch.zeros(rows, dtype=torch.long, device="cuda")
    targets[-3:] = y.cuda()
    logp, lse = f32(rows), f32(rows)
    red.token_logprob_bf16(z, targets, logp, lse)
    want = ref.token_logprob(tail, y, 1.0)
    ref.check("logp", logp[-3:], *want["logp"])
    flat = ref.token_logprob(torch.zeros(1, V), torch.zeros(1, dtype=torch.long), 1.0)["logp"]
    ref.check("logp", logp[:-3], flat[0].expand(rows - 3), flat[1])
    old, adv, rlogp, _ = policy_inputs(tail, y, 1)
    w = torch.zeros(rows, device="cuda")
    w[-3:] = 1.0
    many = lambda v: torch.cat([torch.zeros(rows - 3), v]).cuda()  # noqa: E731
    loss, dz = f32(1), torch.full_like(z, 3.0)
    red.policy_loss_bf16(z, targets, many(old), many(adv), loss, logp, dlogits=dz,
                         ref_logp=many(rlogp), weight=w, kl_coef=0.1)
    want = ref.policy_loss(tail, y, old, adv, torch.ones(3), 1.0, rlogp, kl_coef=0.1)
    ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
    ref.check("dlogits", dz[-3:], *want["dlogits"])
    assert not dz[:-3].any()


@pytest.mark.parametrize("V", [3, 1500])
def test_more_rows_than_one_launch(red, V):
    rows = (1 << 20) + 5
    say("%d rows of %d" % (rows, V))
    z = torch.zeros(rows, V, device="cuda", dtype=torch.bfloat16)
    y = torch.ones(rows, dtype=torch.long, device="cuda")
    logp, lse = f32(rows), f32(rows)
    red.token_logprob_bf16(z, y, logp, lse)
    flat = ref.token_logprob(torch.zeros(1, V), torch.ones(1, dtype=torch.long), 1.0)
    for k, v in (("logp", logp), ("lse", lse)):
        ref.check(k, v, flat[k][0].expand(rows), flat[k][1])
    w = torch.zeros(rows, device="cuda")
    w[0] = w[-1] = 1.0
    loss, dz = f32(1, 2.0), torch.full_like(z, 3.0)
    adv = torch.full_like(w, 0.5)
    red.policy_loss_bf16(z, y, logp, adv, loss, logp.clone(), dlogits=dz, weight=w, accum=True)
    assert abs(loss.item() - 1.0) < 1e-5  # 2 - two rows of ratio 1
    assert dz[0].any() and dz[-1].any() and not dz[1:-1].any()
    g = torch.zeros(rows, device="cuda")
    g[-1] = 1.0
    red.token_logprob_grad_bf16(z, y, lse, g, dz)
    assert dz[-1].any() and not dz[:-1].any()


# --- masks and special values -----------------------------------------------------

@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", [6, 700, 5000, 70001])
def test_masked_logits(red, V, t):
    say("masked logits V=%d %s" % (V, t))
    low = torch.finfo(DTYPES[t]).min
    g, z, y = draw(7, V, t, V)
    z[0, torch.rand(V, generator=g) < 0.7] = -math.inf  # part of a vocabulary
    z[0, y[0]] = 1.0
    z[1, :] = low                                       # one value, the lowest
    z[2, torch.rand(V, generator=g) < 0.7] = low
    z[2, y[2]] = 1.0
    z[3, :] = -math.inf                                 # one column is left
    z[3, y[3]] = -2.0
    z[4, :] = torch.finfo(DTYPES[t]).max
    z[5, :V - 1] = -math.inf                            # the target is masked
    y[5] = 0
    run_logprob(red, z, y, t, 1.0)
    run_logprob(red, z, y, t, 0.5)
    w = torch.ones(7)
    # row 5: ln p = -inf
    keep = torch.tensor([1, 1, 1, 1, 1, 0, 1.0])
    old, adv, rlogp, _ = policy_inputs(z, y, 1)
    run_policy(red, z, y, t, 1, weight=w * keep, ent=0.1, entropy_out=True)
    idx = torch.stack([torch.randperm(V, generator=g)[:4] for _ in range(7)])
    for i in range(7):  # the teacher lists columns that the student has
        have = (z[i] > -math.inf).nonzero().flatten()
        idx[i] = -1
        idx[i, :min(4, len(have))] = have[torch.randperm(len(have), generator=g)[:4]]
    val = torch.randn(7, 4, generator=g)
    run_distill(red, z, idx, val, t, 1.0, w, None)
    run_distill(red, z, idx, val, t, 1.0, torch.tensor([1, 1, 1, 0, 1, 0, 1.0]),
                val.double().logsumexp(1).float() + 0.5)


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("V", [6, 700, 5000, 70001])
def test_bad_rows_stay_alone(red, V, t):
    """NaN, +inf and nothing but -inf make NaN of their own row, and of
    nothing where the row does not count."""
    say("bad rows V=%d %s" % (V, t))
    g, z, y = draw(6, V, t, V)
    z[1, V // 2] = math.nan
    z[3, 0] = math.inf
    z[4, :] = -math.inf
    bad = torch.tensor([0, 1, 0, 1, 1, 0], dtype=torch.bool)
    fine = ~bad
    logp, lse, H = f32(6), f32(6), f32(6)
    getattr(red, "token_logprob_" + t)(z.cuda(), y.cuda(), logp, lse, entropy=H)
    for v in (logp, H):
        assert (v.cpu().isnan() == bad).all(), v
    assert lse[4].item() == -math.inf and lse[1].isnan() and lse[3].isnan()
    want = ref.token_logprob(z[fine], y[fine], 1.0)
    ref.check("logp", logp.cpu()[fine], *want["logp"])
    clean = z.clone()
    clean[bad] = 0.0
    old, adv, rlogp, w = policy_inputs(clean, y, 1)
    w[bad] = 0.0
    idx, val, tl = teacher(clean, 3, 1, True, 1.0)
    starts = torch.tensor([0, 1, 2, 3, 5])  # pair 0: rows 0 and 2; pair 1: rows 1 and 3, 4
    pw = torch.tensor([1.0, 0.0])
    for give in ("weights", "targets"):
        yy, ww = y, w
        if give == "targets":
            yy, ww = torch.where(bad, torch.full_like(y, -100), y), torch.full((6,), 0.5)
        dz = torch.full_like(z, 3.0).cuda()
        loss, lp = f32(1), f32(6)
        getattr(red, "policy_loss_" + t)(z.cuda(), yy.cuda(), old.cuda(), adv.cuda(), loss, lp,
                                         dlogits=dz, ref_logp=rlogp.cuda(), weight=ww.cuda(),
                                         kl_coef=0.1)
        want = ref.policy_loss(clean, yy, old, adv, ww, 1.0, rlogp, kl_coef=0.1)
        ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
        ref.check("logp", lp, *want["logp"])
        ref.check("dlogits", dz, *want["dlogits"])
        assert not dz[bad.cuda()].any()
    for lse_ in (None, tl):
        dz = torch.full_like(z, 3.0).cuda()
        getattr(red, "distill_topk_" + t)(z.cuda(), idx.cuda(), val.cuda(), loss, dlogits=dz,
                                          teacher_lse=cuda(lse_), weight=w.cuda())
        want = ref.distill_topk(clean, idx, val, 1.0, w, lse_)
        ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
        ref.check("dlogits", dz, *want["dlogits"])
    dz = torch.full_like(z, 3.0).cuda()
    seq = f32(4)
    getattr(red, "preference_loss_" + t)(z.cuda(), y.cuda(), starts.cuda(), loss, seq, dlogits=dz,
                                         weight=pw.cuda())
    want = ref.preference_loss(clean, y, starts, pw)
    ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
    ref.check("dlogits", dz, *want["dlogits"])
    # and they do show where they count
    getattr(red, "policy_loss_" + t)(z.cuda(), y.cuda(), old.cuda(), adv.cuda(), loss, lp,
                                     dlogits=dz)
    assert loss.isnan().all() and dz[bad.cuda()].isnan().any(1).all()
    assert not dz[fine.cuda()].isnan().any()


def test_gradient_rows_without_a_factor_are_not_read(red):
    _, z, y = draw(4, 900, "f32", 3)
    z[1] = math.nan
    y[2] = -1
    z[2] = math.nan
    g = torch.tensor([1.0, 0.0, 1.0, -1.0])
    lse = ref.token_logprob(z, y, 1.0)["lse"][0].float()
    dz = torch.full_like(z, 3.0).cuda()
    red.token_logprob_grad_f32(z.cuda(), y.cuda(), lse.cuda(), g.cuda(), dz)
    assert not dz[1:3].any() and dz[0].isfinite().all() and dz[3].any()


# --- the teacher's list -------------------------------------------------------------

@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [9, 1200, 6000, 150000])
def test_teacher_lists(red, V, tail):
    """Padding, entries of no probability, a column listed again, one entry,
    every column, nothing at all."""
    say("teacher lists V=%d tail=%s" % (V, tail))
    g, z, _ = draw(6, V, "f32", V)
    idx, val, lse = teacher(z, 8, 1, tail, 1.0)
    idx[0, 3:] = -1                  # padding
    idx[1, 2], idx[1, 4] = V, 1 << 40  # padding too
    val[2, 1] = -math.inf            # no probability
    idx[3, 5], idx[3, 6] = idx[3, 0], idx[3, 0]  # one column three times
    val[3, 5:7] = val[3, 0] - 1.0
    if tail:
        lse[3] += 2.0                # leaves room for what they add
    idx[4, :] = -1                   # no teacher
    idx[5, :] = torch.tensor([0, V - 1] + [-1] * 6)  # both ends of the row
    w = torch.rand(6, generator=g)
    run_distill(red, z, idx, val, "f32", 1.0, w, lse)
    run_distill(red, z, idx, val, "f32", 1.0, w, lse, shift=3, pad=2)
    run_distill(red, z, idx[:, :1].contiguous(), val[:, :1].contiguous(), "f32", 1.0, w, lse)


@pytest.mark.parametrize("tail", [False, True])
def test_teacher_of_every_column(red, tail):
    g, z, _ = draw(3, 40, "f32", 8)
    t = torch.randn(3, 40, generator=g)
    idx = torch.stack([torch.randperm(40, generator=g) for _ in range(3)])
    lse = t.double().logsumexp(1).float() if tail else None
    run_distill(red, z, idx, t.gather(1, idx), "f32", 1.0, None, lse)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,K", [(1024, 1024), (30000, 1024), (30000, 1000), (262144, 300)])
def test_long_lists_with_a_stride(red, V, K, tail):
    say("lists of %d of %d" % (K, V))
    g, z, _ = draw(2, V, "bf16", V)
    idx, val, lse = teacher(z, K, 1, tail, 0.5)
    wide_i = torch.full((2, K + 3), -7, dtype=torch.long).cuda()
    wide_v = torch.full((2, K + 3), math.nan).cuda()
    wide_i[:, :K], wide_v[:, :K] = idx.cuda(), val.cuda()
    loss, dz = f32(1), torch.empty_like(z).cuda()
    red.distill_topk_bf16(z.cuda(), wide_i[:, :K], wide_v[:, :K], loss, dlogits=dz,
                          teacher_lse=cuda(lse), scale=0.5)
    want = ref.distill_topk(z, idx, val, 0.5, torch.full((2,), 0.5), lse)
    ref.check("loss", loss, want["loss"][0].reshape(1), want["loss"][1])
    ref.check("dlogits", dz, *want["dlogits"])


# --- policies and pairs ---------------------------------------------------------------

def test_policy_branches(red):
    """Both signs of the advantage, below, inside and above the bounds; far
    ratios; no upper bound."""
    n, V = 14, 300
    _, z, y = draw(n, V, "f32", 1)
    logp = ref.token_logprob(z, y, 1.0)["logp"][0].float()
    drift = torch.tensor([-0.5, -0.1, 0.0, 0.1, 0.5, 3.0, -3.0]).repeat(2)
    adv = torch.tensor([1.5] * 7 + [-1.5] * 7)
    w = torch.full((n,), 0.1)
    old = logp - drift
    for high in (0.25, math.inf):
        dz, loss, lp = torch.empty_like(z).cuda(), f32(1, 3.0), f32(n)
        red.policy_loss_f32(z.cuda(), y.cuda(), old.cuda(), adv.cuda(), loss, lp, dlogits=dz,
                            weight=w.cuda(), clip_low=0.2, clip_high=high, accum=True)
        want = ref.policy_loss(z, y, old, adv, w, 1.0, None, 0.2, high)
        ref.check("loss", loss, want["loss"][0].reshape(1) + 3.0, want["loss"][1] + 4 * ref.U)
        ref.check("dlogits", dz, *want["dlogits"])


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("average", [False, True])
def test_ragged_pairs(red, kind, average):
    """Empty sequences, one-row sequences, rows of no sequence, targets that
    do not count, starts outside the rows."""
    n, V = 60, 333
    g, z, y = draw(n, V, "bf16", 5)
    y[4:9] = -100
    starts = torch.tensor([2, 3, 3, 20, 25, 26, 26, 50, 58])
    r = torch.randn(8, generator=g) * 3 - 20.0
    w = torch.tensor([0.5, 0.25, 0.0, 1.0])
    run_preference(red, z, y, "bf16", starts, w, r, kind=kind, beta=0.05, margin=0.3,
                   smoothing=0.1, average=average)
    starts = torch.tensor([-5, 3, 30, 60, 1 << 40])
    run_preference(red, z, y, "bf16", starts, None, r[:4], kind=kind, beta=0.05, average=average)


def test_long_sequences(red):
    """Sums over thousands of rows keep their last bits."""
    n, V = 9001, 64
    g, z, y = draw(n, V, "f32", 6)
    logp = ref.token_logprob(z, y, 1.0)["logp"][0]
    starts = torch.tensor([0, 4000, n])
    r = torch.stack([logp[:4000].sum(), logp[4000:].sum()]).float() + torch.tensor([1.0, -2.0])
    run_preference(red, z, y, "f32", starts, None, r)


# --- accumulation, streams, graphs, repeatability ----------------------------------------

@pytest.mark.parametrize("t", DTYPES)
def test_accum_adds_to_the_old_loss(red, t):
    _, z, y = draw(5, 1000, t, 2)
    old, adv, rlogp, w = policy_inputs(z, y, 2)
    args = (z.cuda(), y.cuda(), old.cuda(), adv.cuda())
    a, b, lp = f32(1), f32(1, 1.5), f32(5)
    getattr(red, "policy_loss_" + t)(*args, a, lp)
    getattr(red, "policy_loss_" + t)(*args, b, lp, accum=True)
    assert abs(b.item() - a.item() - 1.5) <= 4 * ref.U * 2
    idx, val, _ = teacher(z, 3, 1, False, 1.0)
    c, d = f32(1), f32(1, 1.5)
    getattr(red, "distill_topk_" + t)(z.cuda(), idx.cuda(), val.cuda(), c)
    getattr(red, "distill_topk_" + t)(z.cuda(), idx.cuda(), val.cuda(), d, accum=True)
    assert abs(d.item() - c.item() - 1.5) <= 4 * ref.U * 2
    starts = torch.tensor([0, 2, 5]).cuda()
    e, f, seq = f32(1), f32(1, 1.5), f32(2)
    getattr(red, "preference_loss_" + t)(z.cuda(), y.cuda(), starts, e, seq)
    getattr(red, "preference_loss_" + t)(z.cuda(), y.cuda(), starts, f, seq, accum=True)
    assert abs(f.item() - e.item() - 1.5) <= 4 * ref.U * 2


def all_calls(red, s):
    """Every operator once on the tensors of `s`; the outputs."""
    red.token_logprob_bf16(s["z"], s["y"], s["logp"], s["lse"], entropy=s["H"])
    red.token_logprob_grad_bf16(s["z"], s["y"], s["lse"], s["g"], s["d0"], entropy=s["H"],
                                gentropy=s["g"])
    red.distill_topk_bf16(s["z"], s["idx"], s["val"], s["l1"], dlogits=s["d1"],
                          teacher_lse=s["tl"])
    red.policy_loss_bf16(s["z"], s["y"], s["logp"], s["g"], s["l2"], s["lp2"], dlogits=s["d2"],
                         ref_logp=s["g"], kl_coef=0.1, entropy_coef=0.1)
    red.preference_loss_bf16(s["z"], s["y"], s["starts"], s["l3"], s["seq"], dlogits=s["d3"])
    return [s[k] for k in ("logp", "lse", "H", "d0", "l1", "d1", "l2", "lp2", "d2", "l3", "seq",
                           "d3")]


def all_state(rows, V, seed):
    g, z, y = draw(rows, V, "bf16", seed)
    idx, val, tl = teacher(z, 20, 1, True, 1.0)
    s = {"z": z, "y": y, "idx": idx, "val": val, "tl": tl, "g": torch.randn(rows, generator=g) - 8,
         "starts": torch.tensor([0, rows // 4, rows // 2, rows // 2, rows])}
    s = {k: v.cuda() for k, v in s.items()}
    for k in ("logp", "lse", "H", "lp2"):
        s[k] = f32(rows)
    for k in ("l1", "l2", "l3"):
        s[k] = f32(1)
    s["seq"] = f32(4)
    for k in ("d0", "d1", "d2", "d3"):
        s[k] = torch.empty_like(s["z"])
    return s


@pytest.mark.parametrize("rows,V", [(9, 1003), (130, 20000), (7, 140003)])
def test_same_bits_every_time_on_any_stream(red, rows, V):
    say("streams and repeats, %d x %d" % (rows, V))
    s = all_state(rows, V, 3)
    first = [x.clone() for x in all_calls(red, s)]
    for _ in range(3):
        for a, b in zip(first, all_calls(red, s)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    side = torch.cuda.Stream()
    for x in s.values():
        x.record_stream(side)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [x.clone() for x in all_calls(red, s)]
    side.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    red.release_workspace(side)


def test_graph_replays(red):
    s = all_state(40, 5000, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_calls(red, s)  # the workspace is there before the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = all_calls(red, s)
    for seed in (5, 6, 7):
        fresh = all_state(40, 5000, seed)
        for k in ("z", "y", "idx", "val", "tl", "g"):
            s[k].copy_(fresh[k])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        want = all_calls(red, fresh)
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del graph
    red.release_workspace(side)


def test_plans(red):
    s = all_state(6, 3001, 9)
    p = red.plan("policy_loss_bf16", s["z"], s["y"], s["logp"].fill_(-8.0), s["g"], s["l2"],
                 s["lp2"], dlogits=s["d2"])
    q = red.plan("token_logprob_bf16", s["z"], s["y"], s["lp2"].clone(), s["lse"])
    p()
    q()
    a, b = s["l2"].clone(), s["d2"].clone()
    red.policy_loss_bf16(s["z"], s["y"], s["logp"], s["g"], s["l2"], s["lp2"], dlogits=s["d2"])
    assert torch.equal(a, s["l2"]) and torch.equal(b, s["d2"])


# --- gradients against differences of the losses --------------------------------------------

@pytest.mark.parametrize("V", [50, 3001])
def test_gradients_against_differences(red, V):
    """Central differences of the fp32 losses along one direction.  A step of
    2^-6 leaves a third-order term of (2^-6)^2 times the loss's third
    derivative (at most the number of rows in size) and rounding of the loss
    (a few u) over the step."""
    say("differences V=%d" % V)
    rows = 6
    g, z, y = draw(rows, V, "f32", V, std=1.0)
    direction = torch.randn(rows, V, generator=g)
    direction[torch.arange(rows), y] += 1.0
    old, adv, rlogp, w = policy_inputs(z, y, 3)
    old = ref.token_logprob(z, y, 1.0)["logp"][0].float()  # inside the bounds
    idx, val, tl = teacher(z, 5, 2, True, 1.0)
    starts = torch.tensor([0, 3, 6])
    step = 2.0 ** -6

    def policy(zz, dz=None):
        loss, lp = f32(1), f32(rows)
        red.policy_loss_f32(zz.cuda(), y.cuda(), old.cuda(), adv.cuda(), loss, lp, dlogits=dz,
                            ref_logp=rlogp.cuda(), kl_coef=0.1, entropy_coef=0.2)
        return loss.item()

    def distill(zz, dz=None):
        loss = f32(1)
        red.distill_topk_f32(zz.cuda(), idx.cuda(), val.cuda(), loss, dlogits=dz,
                             teacher_lse=tl.cuda())
        return loss.item()

    def preference(zz, dz=None):
        loss, seq = f32(1), f32(2)
        red.preference_loss_f32(zz.cuda(), y.cuda(), starts.cuda(), loss, seq, dlogits=dz)
        return loss.item()

    for loss in (policy, distill, preference):
        dz = torch.empty(rows, V, device="cuda")
        value = loss(z, dz)
        slope = float((dz.cpu().double() * direction.double()).sum())
        up, down = loss(z + step * direction), loss(z - step * direction)
        size = max(1.0, abs(value))
        assert abs((up - down) / (2 * step) - slope) <= step ** 2 * rows * 4 + 8 * ref.U * size / step


# --- what the Python functions refuse -------------------------------------------------------

def test_refused_tensors(red):
    """Shapes, types, strides and devices, with everything else right; the
    calls raise before a kernel runs."""
    s = all_state(4, 100, 1)
    z, y, lp, lse = s["z"], s["y"], s["logp"], s["lse"]
    call = red.token_logprob_bf16
    wide = torch.zeros(4, 200, device="cuda", dtype=torch.bfloat16)
    for bad, why in [
        ((z.float(), y, lp, lse), TypeError), ((z[0], y, lp, lse), ValueError),
        ((wide[:, ::2], y, lp, lse), ValueError), ((z, y[:3], lp, lse), ValueError),
        ((z, y.int(), lp, lse), TypeError), ((z, y.cpu(), lp, lse), ValueError),
        ((z, y, lp.double(), lse), TypeError), ((z, y, wide[:, 0].float()[::2], lse), ValueError),
        ((z, y, lp, None), TypeError), ((z[:1].expand(4, 100), y, lp, lse), ValueError),
    ]:
        with pytest.raises(why):
            call(*bad)
    for kw, why in [(dict(scale=0.0), red.ReduceError), (dict(scale="1"), TypeError),
                    (dict(entropy=lp[:2]), ValueError), (dict(stream="s"), ValueError)]:
        with pytest.raises(why):
            call(z, y, lp, lse, **kw)
    with pytest.raises(ValueError):  # the gradient's shape
        red.token_logprob_grad_bf16(z, y, lse, lp, wide)
    with pytest.raises(ValueError):  # an entropy gradient without the entropy
        red.token_logprob_grad_bf16(z, y, lse, lp, s["d0"], gentropy=lp)
    with pytest.raises(ValueError):
        red.distill_topk_bf16(z, s["idx"][:, :5], s["val"], s["l1"])
    with pytest.raises(ValueError):  # two row strides
        red.distill_topk_bf16(z, s["idx"][:, :5], s["val"][:, :5].contiguous(), s["l1"])
    with pytest.raises(ValueError):
        red.policy_loss_bf16(z, y, lp, lp, s["l2"], s["lp2"], kl_coef=0.1)
    with pytest.raises(ValueError):
        red.preference_loss_bf16(z, y, s["starts"][:4], s["l3"], s["seq"])
    with pytest.raises(ValueError):
        red.preference_loss_bf16(z, y, s["starts"], s["l3"], s["seq"], kind="other")
    with pytest.raises(red.ReduceError):
        red.preference_loss_bf16(z, y, s["starts"], s["l3"], s["seq"], beta=0.0)
    torch.cuda.synchronize()


def test_streams_by_handle_and_object(red):
    s = all_state(5, 700, 2)
    side = torch.cuda.Stream()
    want, got = f32(5), f32(5)
    red.token_logprob_bf16(s["z"], s["y"], want, s["lse"])
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got.zero_()
        torch.cuda.synchronize()
        red.token_logprob_bf16(s["z"], s["y"], got, s["lse"], stream=stream)
        side.synchronize()
        assert torch.equal(got, want)
    plan = red.plan("token_logprob_bf16", s["z"], s["y"], got.zero_(), s["lse"], stream=side)
    torch.cuda.synchronize()
    plan()
    side.synchronize()
    assert torch.equal(got, want)
