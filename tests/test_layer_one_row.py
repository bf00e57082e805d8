"""The operators around the output layer over matrices of one row: its stride is not
looked at.  Without a GPU, on the recorder in place of the HIP runtime."""
import pytest

from test_layer_launch_limits import run  # noqa: F401

STRIDES = [0, 1, 9, (1 << 64) - 1]

CODE = r"""
CALLS["add_rmsnorm"] = [(P, A), (SZ, 1), (SZ, 16), (SZ, "ld"), (P, A + 4096), (SZ, "ld"), (P, A),
    (F, 1e-6), (P, A), (SZ, "ld2"), (P, C), (SZ, "ld"), (P, D_), (SZ, "ld"), (P, A), (P, A),
    (P, None)]
CALLS["rmsnorm_grad"] = [(P, A), (SZ, 1), (SZ, 16), (SZ, "ld"), (P, A), (P, A), (P, A), (SZ, "ld"),
    (P, A), (SZ, "ld"), (P, A), (SZ, "ld2"), (P, C), (I, 0), (P, None)]
CALLS["router_balance"] = [(P, A), (SZ, 1), (SZ, 16), (SZ, "ld"), (P, A), (SZ, 2), (SZ, "ld"), (P, A),
    (F, 0.1), (F, 0.1), (P, B), (I, 0), (P, C), (P, D_), (P, A), (SZ, "ld2"), (P, None)]
CALLS["linear_ce"] = [(P, A), (SZ, 1), (SZ, 16), (SZ, "ld"), (P, A), (SZ, 1), (SZ, "ld"), (P, A),
    (P, A), (F, 1.0), (F, 0.1), (P, B), (I, 0), (P, A), (P, A), (P, C), (SZ, "ld"), (P, D_),
    (SZ, "ld2"), (P, A), (SZ, 1 << 63), (P, None)]
for ld in %r:
    for ld2 in (16, 3):
        print(ld, ld2, *call(%r, %r, ld=ld, ld2=ld2))
"""


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("op", ["add_rmsnorm", "rmsnorm_grad", "router_balance", "linear_ce"])
def test_one_row_has_no_stride(run, op, t):  # noqa: F811
    if (op, t) == ("linear_ce", "f32"):
        pytest.skip("the cross entropy takes 16-bit rows")
    out = run(CODE % (STRIDES, op, t))
    assert len(out) == 2 * len(STRIDES)
    for line in out:
        *_, status, launches, _ = map(int, line.split())
        assert (status, launches > 0) == (0, True), line
