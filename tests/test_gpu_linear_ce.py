"""The output layer's cross entropy and its gradients on the GPU against the
fp64 reference (layer_reference.py), computed on the device in double.

Rows, vocabulary and width sit on both sides of every tile and step; several
device sizes, so that each kind of tile meets ragged edges; hidden rows at any
alignment and stride; masks that leave rows, tiles or everything empty."""
import math

import pytest

import layer_reference as ref
from gpu_helpers import say
from test_gpu_rowloss import DTYPES, place, untouched

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = ["f16", "bf16"]
# (rows, V, D)
SHAPES = [(1, 1, 8), (1, 5, 8), (1, 4097, 1024), (2, 127, 16), (3, 128, 56), (7, 129, 64),
          (31, 1000, 72), (32, 300, 120), (33, 131, 128), (40, 2000, 136), (64, 1023, 192),
          (65, 4096, 200), (100, 255, 8), (127, 257, 320), (128, 999, 512), (129, 640, 72),
          (130, 5001, 1000), (255, 384, 64), (256, 1280, 264), (257, 2049, 328), (500, 3333, 88),
          # rows whose layer is streamed: each group of 16, blocks shared by the waves or
          # not, and widths past the LDS that this takes
          (8, 70, 520), (9, 40000, 24), (16, 3001, 1032), (17, 515, 2056), (48, 1000, 704),
          (49, 33, 1400), (64, 5000, 776), (12, 400, 6152), (60, 300, 2504)]
CASES = [(s, t, cus) for s in SHAPES for t in HALF for cus in (None, 1, 4096)]
BIG = [((1100, 17001, 136), t, None) for t in HALF] + [((2000, 50001, 264), "bf16", None)]


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


def draw(rows, V, D, t, seed, weighted=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    h = (normal(rows, D) * 1.5).to(DTYPES[t])
    W = (normal(V, D) * (1.5 / math.sqrt(D))).to(DTYPES[t])
    y = torch.randint(V, (rows,), device="cuda", generator=g)
    w = None
    if weighted:
        w = torch.rand(rows, device="cuda", generator=g) + 0.25
        w[torch.rand(rows, device="cuda", generator=g) < 0.3] = 0.0
        y[torch.rand(rows, device="cuda", generator=g) < 0.1] = -100
        y[torch.rand(rows, device="cuda", generator=g) < 0.05] = V
        w[rows // 2], y[rows // 2] = 1.0, V - 1
    return h, W, y, w


def put(x, shift, pad, fill=math.nan):
    """place() for a tensor on the device."""
    rows, D = x.shape
    flat = torch.full((shift + rows * (D + pad) + 8,), fill, dtype=x.dtype, device="cuda")
    view = flat[shift:shift + rows * (D + pad)].view(rows, D + pad)[:, :D]
    view.copy_(x)
    return view, flat


def run(red, h, W, y, w, t, scale=1.0, zc=0.0, dh=True, dw=True, odd=False, old=None, **more):
    """A call, everything around its matrices marked; outputs by name."""
    rows, D = h.shape
    shift, pad, gpad = (1, 3, 5) if odd else (0, 0, 0)
    hd, _ = put(h, shift, pad)
    Wd, _ = put(W, 0, 8 if odd else 0)
    out = {"loss": torch.full((1,), 7.0 if old is None else old, device="cuda"),
           "logp": torch.full((rows,), 7.0, device="cuda"),
           "lse": torch.full((rows,), 7.0, device="cuda"), "dhidden": None, "dweight": None}
    marks = []
    if dh:
        out["dhidden"], flat = put(torch.full_like(h, 7.0), shift, gpad, 5.0)
        marks.append((flat, shift, rows, D, gpad))
    if dw:
        out["dweight"], flat = put(torch.full_like(W, 7.0), shift, gpad, 5.0)
        marks.append((flat, shift, W.shape[0], D, gpad))
    getattr(red, "linear_ce_" + t)(hd, Wd, y, out["loss"], logp=out["logp"], lse=out["lse"],
                                   dhidden=out["dhidden"], dweight=out["dweight"], row_weight=w,
                                   scale=scale, z_coef=zc, accum=old is not None, **more)
    for flat, *rest in marks:
        assert untouched(flat, *rest, 5.0)
    return out


def check(got, want):
    for k, v in got.items():
        if v is not None:
            ref.same(k, v, *want[k])


@pytest.mark.parametrize("shape,t,cus", CASES + BIG)
def test_loss_and_gradients(red, monkeypatch, shape, t, cus):
    rows, V, D = shape
    say("linear_ce %d x %d x %d %s cus %s" % (rows, V, D, t, cus))
    if cus:
        monkeypatch.setenv("RED_TEST_CUS", str(cus))
    h, W, y, w = draw(rows, V, D, t, rows + V + D)
    want = ref.linear_ce(h, W, y, w, 0.75, 0.01)
    got = run(red, h, W, y, w, t, 0.75, 0.01, odd=True)
    check(got, want)
    # each output alone has the same bits
    for dh, dw in ((False, False), (True, False), (False, True)):
        some = run(red, h, W, y, w, t, 0.75, 0.01, dh=dh, dw=dw)
        for k, v in some.items():
            assert v is None or torch.equal(v, got[k]), (k, dh, dw)


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("cus", [8, 9, 10, 12, 13, 16, 17, 18, 21])
@pytest.mark.parametrize("masked", [0, 200])
def test_last_round_of_tiles(red, monkeypatch, cus, t, masked):
    """3 x 6 tiles (2 x 6 of rows that count) on so many units that a last round is
    whole, half or a quarter full, or empty, or the only one."""
    say("last round on %d, %d masked %s" % (cus, masked, t))
    monkeypatch.setenv("RED_TEST_CUS", str(cus))
    h, W, y, w = draw(601, 1400, 136, t, cus)
    y[:masked] = -1
    check(run(red, h, W, y, w, t, 0.5, 0.01, odd=True), ref.linear_ce(h, W, y, w, 0.5, 0.01))


@pytest.mark.parametrize("t", HALF)
def test_without_weights(red, t):
    h, W, y, _ = draw(77, 500, 96, t, 3, weighted=False)
    check(run(red, h, W, y, None, t), ref.linear_ce(h, W, y, None, 1.0, 0.0))


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("rows,V,D", [(20011, 14001, 72), (66000, 4500, 40)])
def test_several_pieces(red, rows, V, D, t):
    """Rows so many that the vocabulary takes more than one piece."""
    say("pieces %d x %d x %d %s" % (rows, V, D, t))
    h, W, y, w = draw(rows, V, D, t, rows)
    got = run(red, h, W, y, w, t, 1.0, 0.001)
    check(got, ref.linear_ce(h, W, y, w, 1.0, 0.001))


@pytest.mark.parametrize("t", HALF)
def test_few_rows_and_several_pieces(red, t):
    """A vocabulary past one piece, whose products are not kept."""
    say("few rows, pieces %s" % t)
    h, W, y, w = draw(3, 600001, 16, t, 4)
    check(run(red, h, W, y, w, t, 1.0, 0.001), ref.linear_ce(h, W, y, w, 1.0, 0.001))


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("V,D", [(70000, 640), (70000, 632), (140000, 648)])
def test_products_kept_or_computed_again(red, t, V, D):
    """On both sides of the width and of the size up to which they are kept."""
    say("kept or not %d x %d %s" % (V, D, t))
    h, W, y, w = draw(1040, V, D, t, 5)
    check(run(red, h, W, y, w, t, 1.0, 0.001), ref.linear_ce(h, W, y, w, 1.0, 0.001))


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("rows", [9, 90, 700])
def test_masked_rows_hold_anything(red, monkeypatch, rows, t):
    if rows == 700:
        monkeypatch.setenv("RED_TEST_CUS", "2")
    h, W, y, w = draw(rows, 1111, 136, t, 8)
    dead = (w == 0) | (y < 0) | (y >= 1111)
    want = run(red, h, W, y, w, t, zc=0.01)
    h[dead] = math.nan
    h[dead.nonzero()[0]] = math.inf
    say("masked rows %d %s" % (rows, t))
    got = run(red, h, W, y, w, t, zc=0.01)
    assert all(torch.equal(got[k], want[k]) for k in got)
    assert (got["logp"][dead] == 0).all() and (got["dhidden"][dead] == 0).all()
    # no row counts at all
    none = run(red, h, W, y, torch.zeros_like(w), t, old=1.5)
    assert none["loss"] == 1.5
    assert all((none[k] == 0).all() for k in ("logp", "lse", "dhidden", "dweight"))
    # one row, anywhere
    for at in (0, rows - 1):
        one = torch.zeros_like(w)
        one[at], y[at], h[at] = 2.0, 5, 1.0
        check(run(red, h, W, y, one, t), ref.linear_ce(h, W, y, one, 1.0, 0.0))


@pytest.mark.parametrize("t", HALF)
def test_nan_and_infinity_that_count(red, t):
    h, W, y, w = draw(150, 700, 64, t, 9)
    w[:] = 1.0
    y.clamp_(0, 699)
    want = ref.linear_ce(h, W, y, w, 1.0, 0.0)
    h[5, 3], h[77] = math.nan, math.inf
    say("nan rows %s" % t)
    got = run(red, h, W, y, w, t)
    bad = torch.zeros(150, dtype=torch.bool, device="cuda")
    bad[[5, 77]] = True
    for k in ("logp", "lse", "dhidden"):
        assert got[k][bad].isnan().all(), k
        ref.same(k, got[k][~bad], want[k][0][~bad], want[k][1][~bad])
    assert got["loss"].isnan() and got["dweight"].isnan().all()


@pytest.mark.parametrize("t", HALF)
def test_weights_of_all_sizes(red, t):
    """Factors from 2^-20 to 2^10: half precision keeps each row's gradient."""
    h, W, y, w = draw(140, 900, 128, t, 10)
    y.clamp_(0, 899)
    w = 2.0 ** torch.linspace(-20, 10, 140, device="cuda") * torch.where(
        torch.arange(140, device="cuda") % 3 == 0, -1.0, 1.0)
    say("weights %s" % t)
    check(run(red, h, W, y, w, t, zc=0.05), ref.linear_ce(h, W, y, w, 1.0, 0.05))


@pytest.mark.parametrize("t", HALF)
def test_more_rows_than_one_workgroup_counts(red, t):
    """Rows on both sides of the number up to which each workgroup finds its own
    row's place."""
    for rows in (1024, 1025, 2048, 5000):
        say("places of %d rows %s" % (rows, t))
        h, W, y, w = draw(rows, 130, 32, t, rows)
        check(run(red, h, W, y, w, t), ref.linear_ce(h, W, y, w, 1.0, 0.0))


@pytest.mark.parametrize("t", HALF)
def test_confident_and_far_logits(red, t):
    """Rows whose target has nearly all, and whose target has nearly nothing."""
    g = torch.Generator(device="cuda").manual_seed(2)
    V, D = 640, 64
    W = torch.randn(V, D, device="cuda", generator=g).to(DTYPES[t])
    y = torch.randint(V, (90,), device="cuda", generator=g)
    h = (W[y].float() * torch.linspace(-1.5, 1.5, 90, device="cuda").unsqueeze(1)).to(DTYPES[t])
    say("far logits %s" % t)
    check(run(red, h, W, y, None, t), ref.linear_ce(h, W, y, None, 1.0, 0.0))


@pytest.mark.parametrize("t", HALF)
def test_large_logits(red, t):
    """Logits in the thousands: a row's probabilities rest on differences from its
    largest, not on its log-sum-exp, whose fp32 step is 1e-4 and more there."""
    h, W, y, w = draw(200, 800, 64, t, 21)
    h, W = h * 16, W * 128
    y.clamp_(0, 799)
    w[:] = 1.0 / 200
    say("large logits %s" % t)
    check(run(red, h, W, y, w, t, scale=0.5), ref.linear_ce(h, W, y, w, 0.5, 0.0))
    check(run(red, h[:5], W, y[:5], w[:5], t, scale=0.5),
          ref.linear_ce(h[:5], W, y[:5], w[:5], 0.5, 0.0))


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_subnormal_values_are_kept(red, rows):
    """Hidden values below f16's normal range against large weights."""
    h, W, y, _ = draw(rows, 500, 64, "f16", 22, weighted=False)
    h = (h * 2.0 ** -20).to(h.dtype)
    W = (W.float() * 2.0 ** 12).to(W.dtype)
    assert (h.abs().max() < torch.finfo(torch.float16).tiny) and (h != 0).any()
    say("subnormal %d" % rows)
    want = ref.linear_ce(h, W, y, None, 1.0, 0.0)
    assert want["logp"][0].std() > 1e-3  # the values matter
    check(run(red, h, W, y, None, "f16", scale=1.0), want)
    # as weights: what the gradient of the rows is made of
    check(run(red, W[:rows], h[:rows] if rows < 500 else h, y % rows, None, "f16"),
          ref.linear_ce(W[:rows], h, y % rows, None, 1.0, 0.0))


def test_accumulated_loss_and_same_bits(red):
    h, W, y, w = draw(600, 3000, 128, "bf16", 12)
    first = run(red, h, W, y, w, "bf16")
    for _ in range(3):
        again = run(red, h, W, y, w, "bf16")
        assert all(torch.equal(first[k], again[k]) for k in first)
    more = run(red, h, W, y, w, "bf16", old=2.0, dh=False, dw=False)
    assert abs(more["loss"].item() - 2.0 - first["loss"].item()) <= 2.0 ** -20


def test_workspace_of_the_caller(red):
    h, W, y, w = draw(200, 3000, 128, "bf16", 13)
    want = run(red, h, W, y, w, "bf16")
    size = red.linear_ce_workspace(h, W)
    for small in (dict(dhidden=False), dict(dweight=False), dict(dhidden=False, dweight=False)):
        assert red.linear_ce_workspace(h, W, **small) <= size
    room = torch.full((size + 512,), 0xff, dtype=torch.uint8, device="cuda")  # NaN everywhere
    got = run(red, h, W, y, w, "bf16", workspace=room[:size])
    assert all(torch.equal(got[k], want[k]) for k in got)
    assert (room[size:] == 0xff).all()
    with pytest.raises(red.ReduceError) as e:
        run(red, h, W, y, w, "bf16", workspace=room[:size - 256])
    assert e.value.status == red.RED_ERR_SCRATCH
    with pytest.raises(red.ReduceError) as e:
        run(red, h, W, y, w, "bf16", workspace=room[8:size + 8])
    assert e.value.status == red.RED_ERR_ALIGN


def test_plan_stream_and_graph(red):
    """A plan on a side stream, captured and replayed with new inputs."""
    h, W, y, w = draw(300, 2500, 136, "bf16", 14)
    loss = torch.zeros(1, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(W)
    room = torch.empty(red.linear_ce_workspace(h, W), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with pytest.raises(ValueError, match="workspace"):
        red.linear_ce_bf16(h, W, y, loss, stream=s)
    with pytest.raises(ValueError, match="workspace"):
        red.plan("linear_ce_bf16", h, W, y, loss)
    with torch.cuda.stream(s):
        call = red.plan("linear_ce_bf16", h, W, y, loss, dhidden=dh, dweight=dw, row_weight=w,
                        workspace=room)
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for seed in (15, 16, 17):
        h2, _, y2, w2 = draw(300, 2500, 136, "bf16", seed)
        h.copy_(h2)
        y.copy_(y2)
        w.copy_(w2)
        graph.replay()
        torch.cuda.synchronize()
        want = run(red, h, W, y, w, "bf16")
        assert torch.equal(loss, want["loss"]) and torch.equal(dh, want["dhidden"])
        assert torch.equal(dw, want["dweight"])


def test_refusals(red):
    h = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(7, 16, dtype=torch.bfloat16, device="cuda")
    y, loss = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(1, device="cuda")
    f = red.linear_ce_bf16
    for bad in (dict(weight=W[:, :8]), dict(targets=y[:3]), dict(dhidden=W), dict(dweight=h),
                dict(logp=loss), dict(hidden=h[0]), dict(weight=W.t()),
                dict(loss=torch.zeros(2, device="cuda"))):
        args = dict(hidden=h, weight=W, targets=y, loss=loss)
        args.update(bad)
        with pytest.raises(ValueError):
            f(**args)
    for bad in (dict(hidden=h.half()), dict(weight=W.float()), dict(targets=y.int()),
                dict(workspace=loss)):
        args = dict(hidden=h, weight=W, targets=y, loss=loss)
        args.update(bad)
        with pytest.raises(TypeError):
            f(**args)
    odd = torch.zeros(4, 12, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(red.ReduceError) as e:
        f(odd, torch.zeros(7, 12, dtype=torch.bfloat16, device="cuda"), y, loss)
    assert e.value.status == red.RED_ERR_INVALID
    flat = torch.zeros(8 + 7 * 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(red.ReduceError) as e:
        f(h, flat[4:4 + 7 * 16].view(7, 16), y, loss)
    assert e.value.status == red.RED_ERR_ALIGN
