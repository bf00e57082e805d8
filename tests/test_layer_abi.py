"""Refusals of the operators around the output layer, and their empty input:
none of these calls reaches a kernel (pointers are fake integers that are never
dereferenced), so no GPU is needed."""
import math

import pytest

RED_OK, RED_ERR_INVALID, RED_ERR_ALIGN, RED_ERR_SCRATCH = 0, 1, 2, 5
A = 0x7F0000000000
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
OUT = [A + (i << 20) for i in range(1, 9)]  # outputs: places of their own

CALLS = {
    "add_rmsnorm": [("x", A), ("rows", 3), ("D", 8), ("ldx", 8), ("residual", A), ("ldr", 8),
                    ("weight", A), ("eps", 1e-6), ("sum", OUT[0]), ("lds", 8), ("y", OUT[1]),
                    ("ldy", 8), ("y8", OUT[2]), ("ldy8", 8), ("scale8", OUT[3]), ("rstd", OUT[4]),
                    ("stream", None)],
    "rmsnorm_grad": [("h", A), ("rows", 3), ("D", 8), ("ldh", 8), ("weight", A), ("rstd", A),
                     ("dy", A), ("lddy", 8), ("dsum", A), ("ldds", 8), ("dx", OUT[0]),
                     ("lddx", 8), ("dweight", OUT[1]), ("accum", 0), ("stream", None)],
    "router_balance": [("logits", A), ("rows", 3), ("E", 8), ("ld", 8), ("experts", A), ("K", 2),
                       ("ldk", 2), ("weight", A), ("balance_coef", 0.01), ("z_coef", 0.0),
                       ("loss", OUT[0]), ("accum", 0), ("counts", OUT[1]), ("prob", OUT[2]),
                       ("dlogits", OUT[3]), ("ldd", 8), ("stream", None)],
    "linear_ce": [("hidden", A), ("rows", 3), ("D", 8), ("ldh", 8), ("weight", A), ("V", 5),
                  ("ldw", 8), ("targets", A), ("row_weight", A), ("scale", 1.0), ("z_coef", 0.0),
                  ("loss", OUT[0]), ("accum", 0), ("logp", OUT[1]), ("lse", OUT[2]),
                  ("dhidden", OUT[3]), ("lddh", 8), ("dweight", OUT[4]), ("lddw", 8),
                  ("workspace", OUT[5]), ("workspace_bytes", 1 << 40), ("stream", None)],
}
MATRICES = {"add_rmsnorm": {"x", "residual", "sum", "y"},
            "rmsnorm_grad": {"h", "dy", "dsum", "dx"},
            "router_balance": {"logits", "dlogits"},
            "linear_ce": {"hidden", "weight", "dhidden", "dweight"}}
TYPED = {"add_rmsnorm": {"weight"}, "rmsnorm_grad": {"weight"}, "router_balance": set(),
         "linear_ce": set()}
REQUIRED = {"add_rmsnorm": ["x", "weight"],
            "rmsnorm_grad": ["h", "weight", "rstd", "dy", "dx"],
            "router_balance": ["logits", "experts", "loss", "counts"],
            "linear_ce": ["hidden", "weight", "targets", "loss", "workspace"]}
STRIDES = {"add_rmsnorm": {"ldx": "x", "ldr": "residual", "lds": "sum", "ldy": "y", "ldy8": "y8"},
           "rmsnorm_grad": {"ldh": "h", "lddy": "dy", "ldds": "dsum", "lddx": "dx"},
           "router_balance": {"ld": "logits", "ldk": "experts", "ldd": "dlogits"},
           "linear_ce": {"ldh": "hidden", "ldw": "weight", "lddh": "dhidden", "lddw": "dweight"}}
EIGHT = {"experts", "counts", "targets"}
PAIRS = [(c, t) for c in CALLS for t in SIZE if (c, t) != ("linear_ce", "f32")]
EMPTY = {"add_rmsnorm": ["rows", "D"], "rmsnorm_grad": ["rows", "D"],
         "router_balance": ["rows", "E"], "linear_ce": ["rows", "D", "V"]}


@pytest.fixture(scope="module")
def red():
    return pytest.importorskip("fp32_reductions_amd")


def call(red, name, t, **change):
    assert set(change) <= {k for k, _ in CALLS[name]}
    values = [change.get(k, v) for k, v in CALLS[name]]
    return getattr(red.lib(), "red_%s_%s" % (name, t))(*values)


def is_pointer(v):
    return isinstance(v, int) and v >= A


@pytest.mark.parametrize("name,t", PAIRS)
def test_empty_input(red, name, t):
    nothing = {k: None for k, v in CALLS[name] if is_pointer(v)}
    for k in EMPTY[name]:
        assert call(red, name, t, **{k: 0}, **nothing) == RED_OK, k


@pytest.mark.parametrize("name,t", PAIRS)
def test_null_pointers(red, name, t):
    for k in REQUIRED[name]:
        assert call(red, name, t, **{k: None}) == RED_ERR_INVALID, k


@pytest.mark.parametrize("name,t", PAIRS)
def test_strides_and_sizes(red, name, t):
    for k in STRIDES[name]:
        assert call(red, name, t, **{k: 7 if k != "ldk" else 1}) == RED_ERR_INVALID, k
        assert call(red, name, t, **{k: 1 << 63}) == RED_ERR_INVALID, k
    bad = [dict(rows=1 << 63)]
    if "norm" in name:
        bad += [dict(D=16385, **{k: 16385 for k in STRIDES[name]})]
    if name == "router_balance":
        bad += [dict(E=2049, ld=2049, ldd=2049), dict(K=0), dict(K=1025, ldk=1025), dict(K=3),
                dict(rows=1 << 31)]
    if name == "linear_ce":
        bad += [dict(D=7, ldh=8), dict(D=12, ldh=16, ldw=16, lddh=16, lddw=16), dict(ldw=9),
                dict(rows=(1 << 20) + 1), dict(V=(1 << 24) + 1), dict(ldw=(1 << 21) + 8),
                dict(D=(1 << 16) + 8, ldh=1 << 17, ldw=1 << 17, lddh=1 << 17, lddw=1 << 17)]
    for b in bad:
        assert call(red, name, t, **b) == RED_ERR_INVALID, b


@pytest.mark.parametrize("name,t", PAIRS)
def test_numbers(red, name, t):
    bad = {"add_rmsnorm": [dict(eps=v) for v in (-1e-6, math.nan, math.inf)],
           "rmsnorm_grad": [],
           "router_balance": [{k: v} for k in ("balance_coef", "z_coef")
                              for v in (math.nan, math.inf)],
           "linear_ce": [dict(scale=v) for v in (0.0, -1.0, math.nan, math.inf, 1e31, 1e-31)]
           + [dict(z_coef=math.nan), dict(z_coef=-math.inf)]}[name]
    for b in bad:
        assert call(red, name, t, **b) == RED_ERR_INVALID, b


@pytest.mark.parametrize("t", SIZE)
def test_outputs_of_the_norm(red, t):
    for b in (dict(y=None, y8=None, scale8=None), dict(scale8=None), dict(y8=None),
              dict(y=OUT[0]), dict(y8=OUT[1]), dict(y8=OUT[0]), dict(sum=A, lds=9),
              dict(y=A, ldy=9), dict(sum=A, ldr=9)):
        assert call(red, "add_rmsnorm", t, **b) == RED_ERR_INVALID, b
    for k in ("ldh", "lddy", "ldds"):
        assert call(red, "rmsnorm_grad", t, dx=A, **{k: 9}) == RED_ERR_INVALID, k


@pytest.mark.parametrize("t", SIZE)
def test_gradients_over_inputs(red, t):
    assert call(red, "router_balance", t, dlogits=A, ldd=9) == RED_ERR_INVALID
    if t != "f32":
        assert call(red, "linear_ce", t, dhidden=A, hidden=A) == RED_ERR_INVALID
        assert call(red, "linear_ce", t, dweight=A, weight=A) == RED_ERR_INVALID


@pytest.mark.parametrize("name,t", PAIRS)
def test_alignment(red, name, t):
    for k, v in CALLS[name]:
        if not is_pointer(v) or k in ("y8",):
            continue
        if k in MATRICES[name] | TYPED[name]:
            off = SIZE[t] // 2
        else:
            off = 4 if k in EIGHT else 2
        assert call(red, name, t, **{k: v + off}) == RED_ERR_ALIGN, k
        first = CALLS[name][0][0]
        if k != first:  # a null pointer is reported before an alignment
            assert call(red, name, t, **{k: v + off, first: None}) == RED_ERR_INVALID, k
    if name == "linear_ce":
        assert call(red, name, t, weight=A + 8) == RED_ERR_ALIGN
        assert call(red, name, t, workspace=OUT[5] + 128) == RED_ERR_ALIGN


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_workspace_query(red, t):
    import ctypes

    f = getattr(red.lib(), "red_linear_ce_workspace_" + t)
    size = ctypes.c_size_t(7)
    assert f(4, 8, 5, 1, 1, None) == RED_ERR_INVALID
    for empty in ((0, 8, 5), (4, 0, 5), (4, 8, 0)):
        assert f(*empty, 1, 1, ctypes.byref(size)) == RED_OK and size.value == 0
    for bad in ((4, 12, 5), ((1 << 20) + 1, 8, 5), (4, 8, (1 << 24) + 1), (4, (1 << 16) + 8, 5)):
        assert f(*bad, 1, 1, ctypes.byref(size)) == RED_ERR_INVALID, bad


@pytest.mark.parametrize("name,t", PAIRS)
def test_python_arguments(red, name, t):
    """Names, order and defaults of the Python functions, and what a call with
    the wrong ones raises before any tensor is looked at."""
    import inspect

    torch = pytest.importorskip("torch")
    f = getattr(red, "%s_%s" % (name, t))
    assert f.__doc__ and f.__name__ == "%s_%s" % (name, t)
    first = CALLS[name][0][0]
    names = list(inspect.signature(f).parameters)
    assert names[0] == first and names[-1] == "stream"
    need = [k for k, p in inspect.signature(f).parameters.items()
            if p.default is inspect.Parameter.empty]
    assert names[:len(need)] == need
    with pytest.raises(TypeError, match="missing"):
        f(*[None] * (len(need) - 1))
    with pytest.raises(TypeError, match="unexpected"):
        f(*[None] * len(need), nothing=1)
    with pytest.raises(TypeError, match="%s must be a torch.Tensor" % first):
        f(*[None] * len(need))
    with pytest.raises(TypeError, match="%s must be" % first):
        red.plan("%s_%s" % (name, t), *[None] * len(need))
    host = torch.zeros(3, 8, dtype={"f32": torch.float32, "f16": torch.float16,
                                    "bf16": torch.bfloat16}[t])
    with pytest.raises(ValueError, match="device"):
        f(host, *[None] * (len(need) - 1))
