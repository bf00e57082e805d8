"""The cross entropy's widest rows and largest row strides on the GPU: up to 16 hidden
rows stream the layer while they fit a workgroup's LDS, and take tiles where they do
not, so widths sit on both sides of that."""
import pytest

import layer_reference as ref
from gpu_helpers import say
from test_gpu_linear_ce import HALF, check, draw, run
from test_gpu_rowloss import DTYPES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# rows (ldh + 16) + 8192 bytes of LDS, ldh the width to a multiple of 64 in bytes, of
# 159744: the first of each pair fits
SHAPES = [(16, 400, 4672), (16, 400, 4736), (13, 300, 5760), (13, 300, 5888), (13, 300, 8192),
          (2, 600, 37824), (2, 600, 37952), (1, 130, 65536), (2, 130, 65536), (40, 200, 65536),
          (300, 300, 16392)]


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("shape", SHAPES)
def test_wide_rows(red, shape, t):
    rows, V, D = shape
    say("wide %d x %d x %d %s" % (rows, V, D, t))
    h, W, y, w = draw(rows, V, D, t, rows + V + D)
    got = run(red, h, W, y, w, t, 0.75, 0.01, odd=True)
    check(got, ref.linear_ce(h, W, y, w, 0.75, 0.01))
    alone = run(red, h, W, y, w, t, 0.75, 0.01, dh=False, dw=False)
    for k in ("loss", "logp", "lse"):
        assert torch.equal(alone[k], got[k]), k


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("rows,cus", [(5, None), (30, None), (300, None), (300, 2)])
def test_the_largest_stride(red, monkeypatch, rows, cus, t):
    """Rows of the layer 2^21 elements apart: 4 MiB, so 1 GiB from a tile's first row
    to its last."""
    if cus:
        monkeypatch.setenv("RED_TEST_CUS", str(cus))
    V, D, ld = 300, 72, 1 << 21
    say("stride %d rows cus %s %s" % (rows, cus, t))
    h, W, y, w = draw(rows, V, D, t, rows)
    far = torch.empty_strided((V, D), (ld, 1), dtype=DTYPES[t], device="cuda")
    far.copy_(W)
    dfar = torch.empty_strided((V, D), (ld, 1), dtype=DTYPES[t], device="cuda")
    dh, loss = torch.empty_like(h), torch.empty(1, device="cuda")
    getattr(red, "linear_ce_" + t)(h, far, y, loss, dhidden=dh, dweight=dfar, row_weight=w)
    want = run(red, h, W, y, w, t)
    assert torch.equal(loss, want["loss"]) and torch.equal(dh, want["dhidden"])
    assert torch.equal(dfar, want["dweight"])
