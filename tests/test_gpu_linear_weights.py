"""The cross entropy's rows of very different weights on the GPU: what a row adds to
the layer's gradient keeps its own accuracy however small its weight is beside the
largest, and a row's weight touches no other row's gradient."""
import math

import pytest

import layer_reference as ref
from gpu_helpers import say
from rowloss_reference import half_step
from test_gpu_linear_ce import HALF, check, draw, run
from test_gpu_rowloss import DTYPES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("ratio", [0, 3, 4, 8, 12, 16, 20, 26])
@pytest.mark.parametrize("std", [0.1, 0.01])
@pytest.mark.parametrize("rows", [40, 300, 1500])
def test_a_target_of_one_small_weight(red, rows, std, ratio, t):
    """One light row has a target of its own, which no other row gives a probability
    past e^-55: that row of dW is -w h (1 - p) of the light row and next to nothing of the
    others, whose parts count as errors in full.

    The light row's is rounded with d (half a step), with the result (half a step), and
    where a copy of the hidden row carries part of the weight's exponent with that: half
    of f16's smallest step, 2^-25, times 2^3 of the row's value."""
    V, D, own, light = 130, 64, 77, rows // 3
    g = torch.Generator(device="cuda").manual_seed(rows + ratio)
    W = torch.randn(V, D, device="cuda", generator=g) * 0.05
    h = torch.randn(rows, D, device="cuda", generator=g) * std
    # the other rows' logit of the target: -64
    W[:, 0], h[:, 0] = 0.0, 8.0
    W[own, 0], h[light, 0] = -8.0, 0.0
    W, h = W.to(DTYPES[t]), h.to(DTYPES[t])
    y = torch.randint(own, (rows,), device="cuda", generator=g)
    y[light] = own
    w = torch.full((rows,), 2.0 ** 10, device="cuda")
    w[light] = 1.5 * 2.0 ** (9 - ratio)
    say("light row of %d, 2^-%d of the others, std %g %s" % (rows, ratio, std, t))
    got = run(red, h, W, y, w, t)["dweight"][own].double()
    p = torch.softmax(h.double() @ W.double().t(), 1)[:, own]
    p[light] -= 1.0
    term = (w.double() * p).unsqueeze(1) * h.double()
    assert p[torch.arange(rows, device="cuda") != light].max() < math.exp(-55)
    d, want = w[light].double() * p[light], term.sum(0)
    # the logits' and the sum's fp32 errors are some 200 u of p, which is 1 / V
    error = term[light].abs() * half_step(DTYPES[t]) * (1 + 2.0 ** -6)
    error = error + term.abs().sum(0) - term[light].abs()
    if t == "f16":
        error = error + d.abs() * 2.0 ** -22
    ref.same("dweight", got, *ref.rounded(want, error, DTYPES[t]))


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("rows", [140, 1024, 1025, 3000])
@pytest.mark.parametrize("masked", [False, True])
def test_weights_of_all_sizes_in_any_order(red, rows, masked, t):
    """Factors from 2^-24 to 2^10 in random order, some of them 0, some targets not in the
    layer.  The reference's bound on dW has a term for hidden values that vanish
    beside the largest weight; here it is taken out, and 2^-22 of each term's d put in
    its place."""
    h, W, y, w = draw(rows, 900, 128, t, rows + masked)
    g = torch.Generator(device="cuda").manual_seed(rows)
    u = torch.rand(rows, device="cuda", generator=g)
    sign = torch.where(torch.rand(rows, device="cuda", generator=g) < 0.3, -1.0, 1.0)
    w = torch.where(w != 0, 1.0, 0.0 if masked else 1.0) * 2.0 ** (34 * u - 24) * sign
    if not masked:
        y.clamp_(0, 899)
    say("weights of %d rows %s masked %s" % (rows, t, masked))
    want = ref.linear_ce(h, W, y, w, 1.0, 0.05)
    if t == "f16":
        live = (w != 0) & (y >= 0) & (y < 900)
        x = h.double() @ W.double().t()
        lse = x.logsumexp(1, keepdim=True)
        c = ref.f32(0.05)
        d = (x - lse).exp() * (1 + 2 * c * lse)
        d.scatter_add_(1, y.clamp(0, 899).unsqueeze(1), torch.full_like(lse, -1.0))
        d = torch.where(live.unsqueeze(1), d, 0.0)
        most = w.abs().double().max()
        vanished = 2.0 ** -25 * 2 * most * d.abs().sum(0)
        kept = 2.0 ** -22 * (w.abs().double().unsqueeze(1) * d.abs()).sum(0)
        v, b = want["dweight"]
        b = b + ((kept - vanished) * (1 + half_step(DTYPES[t]))).unsqueeze(1)
        assert (b > 0).all()
        want["dweight"] = v, b
    check(run(red, h, W, y, w, t, zc=0.05), want)


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("rows", [12, 200, 1500])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_weight_that_is_no_number(red, rows, bad, t):
    """It makes the loss and its row's gradient no number, and dW, which sums over
    rows; the other rows' gradients are what they are beside a weight of 0."""
    h, W, y, w = draw(rows, 700, 64, t, rows)
    at = rows // 2
    h[at] = h[0]
    say("weight %g of %d rows %s" % (bad, rows, t))
    w[at] = 0.0
    want = run(red, h, W, y, w, t)
    w[at], y[at] = bad, 3
    got = run(red, h, W, y, w, t)
    keep = torch.arange(rows, device="cuda") != at
    for k in ("logp", "lse", "dhidden"):
        assert torch.equal(got[k][keep], want[k][keep]), k
    assert torch.isfinite(got["logp"][at]) and torch.isfinite(got["lse"][at])
    assert not torch.isfinite(got["loss"]) and got["dhidden"][at].isnan().all()
    assert not torch.isfinite(got["dweight"]).any()


@pytest.mark.parametrize("rows", [12, 200])
@pytest.mark.parametrize("top,scale", [(1e30, 1e10), (1e30, 1e-20), (1e-20, 1e-25), (1e-30, 1e20)])
def test_weights_and_scales_past_one_another(red, rows, top, scale):
    """A weight times the scale need not be an fp32 number, where the values that meet
    it are small or large."""
    h, W, y, w = draw(rows, 500, 64, "bf16", rows)
    w = torch.where(w == 0, 0.0, top * 2.0 ** -(torch.arange(rows, device="cuda") % 60).float())
    size = scale ** -0.5
    h, W = (h.double() * size).bfloat16(), (W.double() * size).bfloat16()
    assert h.isfinite().all() and W.isfinite().all()
    say("weight %g scale %g, %d rows" % (top, scale, rows))
    want = ref.linear_ce(h, W, y, w, scale, 0.0)
    assert want["dhidden"][0].abs().max() < 1e37 and want["dweight"][0].abs().max() < 1e37
    check(run(red, h, W, y, w, "bf16", scale=scale), want)


@pytest.mark.parametrize("rows", [300, 1500])
def test_captured_and_replayed_with_other_weights(red, rows):
    """The groups of weights are found anew in every replay: one group, many, none."""
    h, W, y, w = draw(rows, 700, 72, "f16", rows)
    loss, dh, dw = torch.zeros(1, device="cuda"), torch.empty_like(h), torch.empty_like(W)
    room = torch.empty(red.linear_ce_workspace(h, W), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call = red.plan("linear_ce_f16", h, W, y, loss, dhidden=dh, dweight=dw, row_weight=w,
                        workspace=room)
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for span in (0, 30, 3, 90, None, 12):
        say("replay over weights of 2^-%s" % span)
        h2, _, y2, w2 = draw(rows, 700, 72, "f16", rows + (span or 0))
        h.copy_(h2)
        y.copy_(y2)
        w.copy_(torch.zeros_like(w2) if span is None else w2 * 2.0 ** (-span * torch.rand_like(w2)))
        graph.replay()
        torch.cuda.synchronize()
        want = run(red, h, W, y, w, "f16")
        assert torch.equal(loss, want["loss"]) and torch.equal(dh, want["dhidden"])
        assert torch.equal(dw, want["dweight"])
        if span is not None:
            check(want, ref.linear_ce(h, W, y, w, 1.0, 0.0))
