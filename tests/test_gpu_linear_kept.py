"""The cross entropy's products kept for the gradients, and computed again, on both sides
of the number of bytes per width up to which they are kept."""
import pytest

import layer_reference as ref
from gpu_helpers import say
from test_gpu_linear_ce import HALF, check, draw, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


# 4 rows (V to 256) against D 384 KiB: the first of each pair is kept
SHAPES = [(200, 3840, 8), (200, 4096, 8), (90, 52224, 48), (90, 53248, 48), (15, 20000, 8),
          (15, 60000, 8), (333, 18688, 64), (333, 19200, 64), (1025, 61184, 632), (1025, 61000, 640)]


@pytest.mark.parametrize("t", HALF)
@pytest.mark.parametrize("shape", SHAPES)
def test_kept_and_computed_again(red, shape, t):
    rows, V, D = shape
    say("kept %d x %d x %d %s" % (rows, V, D, t))
    h, W, y, w = draw(rows, V, D, t, rows + V + D)
    got = run(red, h, W, y, w, t, 0.75, 0.01)
    check(got, ref.linear_ce(h, W, y, w, 0.75, 0.01))
    # The workspace has d either way; the rest but for the products takes less than they.
    columns = -(-V // 256) * 256
    kept, d = 4 * rows * columns, 2 * columns * (-(-rows // 256) * 256)
    size = red.linear_ce_workspace(h, W) - red.linear_ce_workspace(h, W, False, False)
    assert (size >= kept + d) == (D >= 640 or kept <= D * 384 * 1024)
