"""A router's balance loss, counts and gradient on the GPU against the fp64
reference (layer_reference.py)."""
import math

import pytest

import layer_reference as ref
from gpu_helpers import say
from test_gpu_rowloss import DTYPES, place, untouched

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# experts on both sides of each number of lanes and vectors a row is given, in
# one workgroup and in many
EXPERTS = [1, 2, 3, 7, 8, 15, 16, 17, 31, 32, 33, 61, 64, 127, 128, 129, 255, 256, 257, 511, 512,
           513, 1000, 1024, 1025, 2047, 2048]
CASES = [(rows, E, t) for i, E in enumerate(EXPERTS) for rows in (1, 13, 1027 + 50 * i)
         for t in DTYPES] + [(70001, E, t) for E in (8, 61, 128) for t in DTYPES]


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


def draw(rows, E, K, t, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(rows, E, generator=g) * std + torch.randn(E, generator=g)).to(DTYPES[t])
    experts = torch.rand(rows, E, generator=g).topk(min(K, E), dim=1).indices
    w = torch.rand(rows, generator=g) + 0.5
    w[torch.rand(rows, generator=g) < 0.3] = 0.0
    return g, z, experts.contiguous(), w


def run(red, z, experts, w, t, balance=0.02, zc=0.003, grad=True, shift=0, pad=0, old=None, **more):
    rows, E = z.shape
    loss = torch.full((1,), 7.0 if old is None else old, device="cuda")
    counts = torch.full((E,), -1, dtype=torch.int64, device="cuda")
    prob = torch.full((E,), 9.0, device="cuda")
    zd, _ = place(z, shift, pad)
    dz, flat = place(torch.full_like(z, 7.0), shift, pad, 5.0) if grad else (None, None)
    getattr(red, "router_balance_" + t)(
        zd, experts.cuda(), loss, counts, dlogits=dz, weight=None if w is None else w.cuda(),
        prob=prob, balance_coef=balance, z_coef=zc, accum=old is not None, **more)
    if grad:
        assert untouched(flat, shift, rows, E, pad, 5.0)
    return {"loss": loss, "counts": counts, "prob": prob, "dlogits": dz}


def check(got, want):
    for k, v in got.items():
        if v is not None:
            ref.same(k, v, *want[k])


@pytest.mark.parametrize("rows,E,t", CASES)
def test_loss_counts_and_gradient(red, rows, E, t):
    say("router %d x %d %s" % (rows, E, t))
    K = 1 + E % 7
    _, z, experts, w = draw(rows, E, K, t, rows + E)
    shift, pad = (1, 3) if E % 2 else (0, 8)
    got = run(red, z, experts, w, t, shift=shift, pad=pad)
    check(got, ref.router_balance(z, experts, w, 0.02, 0.003))
    alone = run(red, z, experts, w, t, grad=False)
    assert torch.equal(alone["loss"], got["loss"]) or shift or pad
    check(run(red, z, experts, None, t, zc=0.0), ref.router_balance(z, experts, None, 0.02, 0.0))


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows", [40, 5000])
def test_masks(red, rows, t):
    """Rows that do not count hold anything; padded and repeated choices."""
    E = 48
    g, z, experts, w = draw(rows, E, 4, t, 3)
    experts[::3, 1] = -1
    experts[1::3, 2] = E
    experts[2::3, 3] = experts[2::3, 0]
    experts[0, 0], experts[1, 0] = 1 << 62, -(1 << 62)
    w[0], w[1], w[3] = 1.0, 0.5, 0.0
    want = ref.router_balance(z, experts, w, 0.02, 0.003)
    z[w == 0] = math.nan
    say("router masks %d %s" % (rows, t))
    got = run(red, z, experts, w, t)
    check(got, want)
    assert (got["dlogits"][(w == 0).cuda()] == 0).all()
    # nothing counts; nothing is chosen
    none = run(red, z, experts, torch.zeros(rows), t, old=3.0)
    assert none["loss"] == 3.0 and (none["counts"] == 0).all() and (none["prob"] == 0).all()
    assert (none["dlogits"] == 0).all()
    z = torch.where(z.isnan(), torch.zeros_like(z), z)
    check(run(red, z, torch.full_like(experts, -1), w, t),
          ref.router_balance(z, torch.full_like(experts, -1), w, 0.02, 0.003))


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows", [30, 4000])
def test_infinities_and_nan(red, rows, t):
    E = 20
    _, z, experts, w = draw(rows, E, 2, t, 4)
    w[:4] = 1.0
    z[::5, 3] = -math.inf
    z[1::5, :19] = torch.finfo(z.dtype).min / 4
    say("router -inf %d %s" % (rows, t))
    check(run(red, z, experts, w, t), ref.router_balance(z, experts, w, 0.02, 0.003))
    want = ref.router_balance(z, experts, w, 0.02, 0.0)["dlogits"]
    z[0, 2], z[2, 1], z[3] = math.nan, math.inf, -math.inf
    got = run(red, z, experts, w, t, zc=0.0)
    bad = torch.zeros(rows, dtype=torch.bool)
    bad[[0, 2, 3]] = True
    assert got["dlogits"][bad.cuda()].isnan().all() and got["loss"].isnan()
    ref.same("dlogits", got["dlogits"].cpu()[~bad], want[0][~bad], want[1][~bad])


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows", [50, 6000])
def test_in_place_accumulated_and_strided_choices(red, rows, t):
    E = 64
    _, z, experts, w = draw(rows, E, 6, t, 5)
    want = run(red, z, experts, w, t)
    zd, loss = z.cuda(), torch.full((1,), 2.5, device="cuda")
    counts = torch.empty(E, dtype=torch.int64, device="cuda")
    wide = torch.full((rows, 9), 5, device="cuda")
    wide[:, :6] = experts.cuda()
    say("router in place %d %s" % (rows, t))
    getattr(red, "router_balance_" + t)(zd, wide[:, :6], loss, counts, dlogits=zd,
                                        weight=w.cuda(), balance_coef=0.02, z_coef=0.003,
                                        accum=True)
    assert torch.equal(zd, want["dlogits"]) and torch.equal(counts, want["counts"])
    v, b = ref.router_balance(z, experts, w, 0.02, 0.003)["loss"]
    ref.same("loss", loss, v + 2.5, b + 2.0 ** -22)


def test_same_bits_again(red):
    _, z, experts, w = draw(30011, 96, 6, "bf16", 9)
    first = run(red, z, experts, w, "bf16")
    for _ in range(3):
        again = run(red, z, experts, w, "bf16")
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_refusals(red):
    z = torch.zeros(4, 8, device="cuda")
    e = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    loss, counts = torch.zeros(1, device="cuda"), torch.zeros(8, dtype=torch.int64, device="cuda")
    f = red.router_balance_f32
    for bad in (dict(experts=e[:3]), dict(counts=counts[:7]), dict(loss=torch.zeros(2, device="cuda")),
                dict(dlogits=z[:, :4]), dict(weight=torch.zeros(3, device="cuda")),
                dict(experts=e.t()), dict(logits=z[0])):
        args = dict(logits=z, experts=e, loss=loss, counts=counts)
        args.update(bad)
        with pytest.raises(ValueError):
            f(**args)
    for bad in (dict(experts=e.int()), dict(counts=counts.int()), dict(logits=z.half())):
        args = dict(logits=z, experts=e, loss=loss, counts=counts)
        args.update(bad)
        with pytest.raises(TypeError):
            f(**args)
    with pytest.raises(red.ReduceError):
        f(z, e[:, :0], loss, counts)
    wide = torch.zeros(2, 2049, device="cuda")
    with pytest.raises(red.ReduceError):
        f(wide, e[:2], loss, torch.zeros(2049, dtype=torch.int64, device="cuda"))
