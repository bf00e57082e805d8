"""The norm's weight gradient over many rows of each workgroup on the GPU: its error
does not grow with their number."""
import math

import pytest

import layer_reference as ref
from gpu_helpers import say
from rowloss_reference import U
from test_gpu_rowloss import DTYPES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


# (rows, width), each number of threads and vectors that a row is given
SHAPES = [(200003, 8), (60001, 61), (40000, 256), (40000, 500), (20000, 1000), (6000, 4100),
          (1600, 9000), (1600, 16384)]


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("accum", [False, True])
def test_column_sums_of_many_rows(red, monkeypatch, rows, D, t, accum):
    """On one compute unit, so that a workgroup takes most of the rows.  Every term of a
    column is 1 + e, e just under half an fp32 step of the last sums: added one after
    another in fp32 the last ones would all lose their e.

    A term is two products (2 u); 64 of them at most follow each other in fp32, 16 of
    a workgroup's rows may meet so, a workgroup's sum is rounded once and the result is:
    84 u."""
    monkeypatch.setenv("RED_TEST_CUS", "1")
    # Lanes that share a column: the longest chain is rows over them.
    vecs = -(-D // (4 if t == "f32" else 8))
    sharing = 64 if vecs <= 16 else 16 if vecs <= 128 else max(1, 1024 // (-(-vecs // 64) * 64))
    e = 0.99 * 2.0 ** (math.floor(math.log2(rows / sharing)) - 24)
    say("column sums %d x %d %s" % (rows, D, t))
    h = torch.ones(rows, D, dtype=DTYPES[t], device="cuda")
    rstd = torch.full((rows,), 1.0 + e, device="cuda")
    w = torch.ones(D, dtype=DTYPES[t], device="cuda")
    dw = torch.full((D,), 3.0, device="cuda")
    getattr(red, "rmsnorm_grad_" + t)(h, w, rstd, h, torch.empty_like(h), dweight=dw, accum=accum)
    want = rows * rstd[0].double() + (3.0 if accum else 0.0)
    ref.same("dweight", dw, want.expand(D), 84 * U * want)


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows,D", [(5000, 40), (3001, 260), (3000, 520), (700, 2056), (300, 16384)])
def test_gradient_of_many_rows(red, monkeypatch, rows, D, t):
    """Ordinary rows in the same number of steps, added to old values, all outputs."""
    monkeypatch.setenv("RED_TEST_CUS", "1")
    g = torch.Generator(device="cuda").manual_seed(rows + D)

    def matrix(std):
        return (torch.randn(rows, D, device="cuda", generator=g) * std).to(DTYPES[t])

    h, dy, ds = matrix(2.0), matrix(0.1), matrix(0.1)
    w = matrix(1.0)[0].contiguous()
    rstd = (h.double().square().mean(1) + 1e-5).rsqrt().float()
    old = torch.randn(D, device="cuda", generator=g)
    say("many rows %d x %d %s" % (rows, D, t))
    dx, dw = torch.empty_like(h), old.clone()
    f = getattr(red, "rmsnorm_grad_" + t)
    f(h, w, rstd, dy, dx, dsum=ds, dweight=dw, accum=True)
    want = ref.rmsnorm_grad(h, w, rstd, dy, ds)
    ref.same("dx", dx, *want["dx"])
    n = h.double() * rstd.double().unsqueeze(1)
    terms = (dy.double() * n).abs().sum(0)
    v = want["dweight"][0] + old.double()
    ref.same("dweight", dw, v, 84 * U * terms + U * (v.abs() + old.abs()))
    again = old.clone()
    f(h, w, rstd, dy, dx, dsum=ds, dweight=again, accum=True)
    assert torch.equal(again, dw)
