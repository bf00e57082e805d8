"""What a row with an infinity gives in the norm and its gradient on the GPU, as
include/reduce.h has it: rstd 0, NaN at the infinities, zeros elsewhere, scale 0; a
gradient of NaN; and nothing in any other row."""
import math

import pytest

import layer_reference as ref
from gpu_helpers import say
from test_gpu_rowloss import DTYPES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("t", DTYPES)
@pytest.mark.parametrize("rows,D", [(3, 40), (6, 777), (700, 264), (300, 9000)])
@pytest.mark.parametrize("where", ["x", "residual", "sum"])
def test_infinity(rows, D, t, where):
    import fp32_reductions_amd as red

    if where == "sum" and t == "f16":
        pytest.skip("two finite f16 values have a finite fp32 sum")
    say("infinity in %s %d x %d %s" % (where, rows, D, t))
    g = torch.Generator().manual_seed(rows)
    x, r, dy = ((torch.randn(rows, D, generator=g) * 2).to(DTYPES[t]) for _ in range(3))
    w = torch.randn(D, generator=g).to(DTYPES[t])

    def run():
        h, y = (torch.empty(rows, D, dtype=DTYPES[t], device="cuda") for _ in range(2))
        y8 = torch.empty(rows, D, dtype=ref.E4M3, device="cuda")
        scale, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        getattr(red, "add_rmsnorm_" + t)(x.cuda(), w.cuda(), y, residual=r.cuda(), sum=h, y8=y8,
                                         yscale=scale, rstd=rstd)
        dx = torch.empty_like(h)
        getattr(red, "rmsnorm_grad_" + t)(h, w.cuda(), rstd, dy.cuda(), dx)
        return {"h": h, "y": y, "y8": y8.float(), "scale": scale, "rstd": rstd, "dx": dx}

    want = run()
    bad, at = rows // 2, [3, D - 1]
    most = torch.finfo(DTYPES[t]).max
    if where == "sum":
        x[bad, at] = r[bad, at] = most
    else:
        (x if where == "x" else r)[bad, at] = -math.inf
    got = run()
    keep = torch.arange(rows, device="cuda") != bad
    for k in want:
        assert torch.equal(got[k][keep], want[k][keep]), k
    hit = torch.zeros(D, dtype=torch.bool, device="cuda")
    hit[at] = True
    assert got["h"][bad][hit].isinf().all() and got["h"][bad][~hit].isfinite().all()
    assert got["rstd"][bad] == 0 and got["scale"][bad] == 0
    for k in ("y", "y8"):
        assert got[k][bad][hit].isnan().all() and (got[k][bad][~hit] == 0).all(), k
    assert got["dx"][bad].isnan().all()
