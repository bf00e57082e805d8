"""The router's balance loss without its gradient on the GPU: a launch of its own,
and the same results as beside a gradient, bit for bit."""
import pytest

import layer_reference as ref
from gpu_helpers import say
from test_gpu_router import EXPERTS, check, draw, run
from test_gpu_rowloss import DTYPES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("rows", [13, 1200])
@pytest.mark.parametrize("weighted", [False, True])
def test_loss_alone(red, rows, E, t, weighted):
    say("router alone %d x %d %s" % (rows, E, t))
    _, z, experts, w = draw(rows, E, 1 + E % 7, t, rows + E)
    w = w if weighted else None
    shift, pad = (1, 3) if E % 2 else (0, 8)
    both = run(red, z, experts, w, t, shift=shift, pad=pad)
    alone = run(red, z, experts, w, t, grad=False, shift=shift, pad=pad)
    for k in ("loss", "counts", "prob"):
        assert torch.equal(alone[k], both[k]), k
    check(alone, ref.router_balance(z, experts, w, 0.02, 0.003))


@pytest.mark.parametrize("t", DTYPES)
def test_loss_alone_of_many_rows_added(red, t):
    say("router alone, added %s" % t)
    _, z, experts, w = draw(70001, 61, 4, t, 21)
    both = run(red, z, experts, w, t, old=2.5)
    alone = run(red, z, experts, w, t, old=2.5, grad=False)
    for k in ("loss", "counts", "prob"):
        assert torch.equal(alone[k], both[k]), k
