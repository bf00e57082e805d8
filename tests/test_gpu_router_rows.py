"""The router's sums over many rows of each workgroup on the GPU: their error does not
grow with the rows."""
import math

import pytest

import layer_reference as ref
from gpu_helpers import say
from rowloss_reference import U
from test_gpu_router import check, draw, run
from test_gpu_rowloss import DTYPES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("E", [8, 64, 128, 256, 512, 1024, 2048])
@pytest.mark.parametrize("grad", [False, True])
def test_probabilities_of_many_rows(red, monkeypatch, E, t, grad):
    """On one compute unit.  Every row's p is 1 / E and its weight 1 + e, e just under half
    an fp32 step of the last sums: added one after another in fp32 the last ones would
    all lose their e.

    The logits are 0: p is exact.  A term is a quotient and a product (2 u), 256 at most
    follow each other in fp32, 10 more join lanes and 16 waves, the rest is fp64: 284 u.
    The loss is b E sum f P of the same P, and the gradients are 0 but for
    rounding (p q and its sum over E, which are E equal values)."""
    monkeypatch.setenv("RED_TEST_CUS", "1")
    vecs = -(-E // (4 if t == "f32" else 8))
    lanes = 4 if vecs <= 4 else 16 if vecs <= 32 else 64
    terms = 4000
    rows = terms * (1024 // lanes) + 3
    e = 0.99 * 2.0 ** (math.floor(math.log2(terms)) - 24)
    say("router sums %d x %d %s" % (rows, E, t))
    z = torch.zeros(rows, E, dtype=DTYPES[t], device="cuda")
    experts = (torch.arange(rows, device="cuda") % E).unsqueeze(1)
    w = torch.full((rows,), 1.0 + e, device="cuda")
    loss, prob = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
    counts = torch.empty(E, dtype=torch.int64, device="cuda")
    dz = torch.full_like(z, 7.0) if grad else None
    getattr(red, "router_balance_" + t)(z, experts, loss, counts, dlogits=dz, weight=w, prob=prob,
                                        balance_coef=1.0, z_coef=0.0)
    assert torch.equal(counts, torch.bincount(experts.reshape(-1), minlength=E))
    want = rows * w[0].double() / E
    ref.same("prob", prob, want.expand(E), 284 * U * want)
    ref.same("loss", loss, (want * E).reshape(1), 284 * U * want * E)
    if grad:
        f = counts.double() * E / rows
        value = w[0].double() / E * (f - f.mean())
        ref.same("dlogits", dz, value.expand(rows, E),
                 ref.rounded(value, w[0].double() / E * (E + 10) * U * f.max(), z.dtype)[1])


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("E", [6, 100, 700])
def test_ordinary_rows(red, monkeypatch, E, t):
    """More rows than one step of the sums takes, masked rows among them, with all outputs,
    on devices of one and of two units; each again with the same bits."""
    vecs = -(-E // (4 if t == "f32" else 8))
    lanes = 4 if vecs <= 4 else 16 if vecs <= 32 else 64
    rows = 2 * 256 * (1024 // lanes) + 77
    _, z, experts, w = draw(rows, E, 3, t, E)
    w[256 * (1024 // lanes):][:100] = 0.0
    want = ref.router_balance(z, experts, w, 0.02, 0.003)
    for cus in (1, 2):
        monkeypatch.setenv("RED_TEST_CUS", str(cus))
        say("router %d x %d %s cus %d" % (rows, E, t, cus))
        got = run(red, z, experts, w, t)
        check(got, want)
        again = run(red, z, experts, w, t)
        assert all(torch.equal(got[k], again[k]) for k in got)
        added = run(red, z, experts, w, t, old=3.0, grad=False)
        assert torch.equal(added["prob"], got["prob"]) and torch.equal(added["counts"], got["counts"])


def test_captured_and_replayed(red, monkeypatch):
    """Several launches of the sums in a graph, replayed with new rows."""
    monkeypatch.setenv("RED_TEST_CUS", "1")
    rows, E = 3 * 256 * 64 + 5, 48
    say("router replays")
    _, z, experts, w = draw(rows, E, 2, "bf16", 1)
    zd, ed, wd = z.cuda(), experts.cuda(), w.cuda()
    loss, prob = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
    counts = torch.empty(E, dtype=torch.int64, device="cuda")
    dz = torch.empty_like(zd)

    def call():
        red.router_balance_bf16(zd, ed, loss, counts, dlogits=dz, weight=wd, prob=prob,
                                balance_coef=0.02, z_coef=0.003)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for seed in (2, 3, 4):
        _, z2, e2, w2 = draw(rows, E, 2, "bf16", seed)
        for old, new in ((zd, z2), (ed, e2), (wd, w2)):
            old.copy_(new)
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        got = [v.clone() for v in (loss, counts, prob, dz)]
        want = run(red, z2, e2, w2, "bf16")
        torch.cuda.synchronize()
        assert all(torch.equal(a, want[k]) for a, k in zip(got, ("loss", "counts", "prob", "dlogits")))
        check(want, ref.router_balance(z2, e2, w2, 0.02, 0.003))
