"""Refusals of the losses over rows of logits, and their empty input: none of
these calls reaches a kernel (pointers are fake integers that are never
dereferenced), so no GPU is needed."""
import ctypes
import math
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBRARY = os.path.join(ROOT, "fp32_reductions_amd", "libreduce.so")
RED_OK, RED_ERR_INVALID, RED_ERR_ALIGN = 0, 1, 2
A = 0x7F0000000000
SIZE = {"f32": 4, "f16": 2, "bf16": 2}

# Arguments of each call in order, with values that pass.
MATRIX = [("logits", A), ("rows", 3), ("V", 5), ("ld", 5)]
CALLS = {
    "token_logprob": MATRIX + [("targets", A), ("scale", 1.0), ("logp", A), ("lse", A),
                               ("entropy", A), ("stream", None)],
    "token_logprob_grad": MATRIX + [("targets", A), ("scale", 1.0), ("lse", A), ("entropy", A),
                                    ("glogp", A), ("gentropy", A), ("dlogits", A + 4096),
                                    ("ldd", 5), ("stream", None)],
    "distill_topk": MATRIX + [("idx", A), ("val", A), ("K", 2), ("ldk", 2), ("teacher_lse", A),
                              ("weight", A), ("scale", 1.0), ("loss", A), ("accum", 0),
                              ("row_loss", A), ("dlogits", A + 4096), ("ldd", 5),
                              ("stream", None)],
    "policy_loss": MATRIX + [("targets", A), ("old_logp", A), ("ref_logp", A), ("advantage", A),
                             ("weight", A), ("scale", 1.0), ("clip_low", 0.2), ("clip_high", 0.2),
                             ("kl_coef", 0.1), ("entropy_coef", 0.0), ("loss", A), ("accum", 0),
                             ("logp", A), ("entropy", A), ("dlogits", A + 4096), ("ldd", 5),
                             ("stream", None)],
    "preference_loss": MATRIX + [("targets", A), ("starts", A), ("pairs", 1), ("ref_logp", A),
                                 ("weight", A), ("kind", 0), ("beta", 0.1), ("margin", 0.0),
                                 ("smoothing", 0.0), ("average", 0), ("loss", A), ("accum", 0),
                                 ("seq_logp", A), ("dlogits", A + 4096), ("ldd", 5),
                                 ("stream", None)],
}
REQUIRED = {
    "token_logprob": ["logits", "targets", "logp", "lse"],
    "token_logprob_grad": ["logits", "targets", "lse", "glogp", "dlogits", "entropy"],
    "distill_topk": ["logits", "idx", "val", "loss"],
    "policy_loss": ["logits", "targets", "old_logp", "ref_logp", "advantage", "loss", "logp"],
    "preference_loss": ["logits", "targets", "starts", "loss", "seq_logp"],
}
INT64 = {"targets", "idx", "starts"}
PAIRS = [(c, t) for c in CALLS for t in SIZE]


@pytest.fixture(scope="module")
def red():
    return pytest.importorskip("fp32_reductions_amd")


def call(red, name, t, **change):
    values = [change.get(k, v) for k, v in CALLS[name]]
    assert set(change) <= {k for k, _ in CALLS[name]}
    return getattr(red.lib(), "red_%s_%s" % (name, t))(*values)


@pytest.mark.parametrize("name,t", PAIRS)
def test_empty_input(red, name, t):
    nothing = {k: None for k, v in CALLS[name] if v == A or v == A + 4096}
    assert call(red, name, t, rows=0, **nothing) == RED_OK
    assert call(red, name, t, V=0, **nothing) == RED_OK
    if name == "preference_loss":
        assert call(red, name, t, pairs=0, **nothing) == RED_OK


@pytest.mark.parametrize("name,t", PAIRS)
def test_null_pointers(red, name, t):
    for k in REQUIRED[name]:
        assert call(red, name, t, **{k: None}) == RED_ERR_INVALID, k


@pytest.mark.parametrize("name,t", PAIRS)
def test_sizes(red, name, t):
    bad = [dict(ld=4), dict(V=1 << 31, ld=1 << 31), dict(rows=1 << 40, ld=1 << 40),
           dict(rows=(1 << 64) - 1)]
    if name != "token_logprob":
        bad += [dict(ldd=4), dict(ldd=1 << 63), dict(dlogits=A, ldd=6)]
    if name == "distill_topk":
        bad += [dict(K=0), dict(K=1025, ldk=1025), dict(K=3), dict(ldk=1 << 62),
                dict(V=393217, ld=393217, ldd=393217)]
    if name == "preference_loss":
        bad += [dict(rows=(1 << 19) + 1), dict(pairs=(1 << 17) + 1)]
    for b in bad:
        assert call(red, name, t, **b) == RED_ERR_INVALID, b


@pytest.mark.parametrize("name,t", PAIRS)
def test_numbers(red, name, t):
    bad = []
    if name != "preference_loss":
        bad += [dict(scale=v) for v in (0.0, -1.0, math.nan, math.inf, 1e31, 1e-31)]
    if name == "policy_loss":
        bad += [dict(clip_low=-0.1), dict(clip_high=-0.1), dict(clip_low=math.nan),
                dict(clip_high=math.nan), dict(kl_coef=math.inf), dict(entropy_coef=math.nan)]
    if name == "preference_loss":
        bad += [dict(kind=-1), dict(kind=3), dict(beta=0.0), dict(beta=-1.0), dict(beta=math.nan),
                dict(beta=math.inf), dict(margin=math.inf), dict(smoothing=-0.1),
                dict(smoothing=1.5), dict(smoothing=math.nan)]
    for b in bad:
        assert call(red, name, t, **b) == RED_ERR_INVALID, b


@pytest.mark.parametrize("name,t", PAIRS)
def test_alignment(red, name, t):
    for k, v in CALLS[name]:
        if v != A and v != A + 4096:
            continue
        need = SIZE[t] if k in ("logits", "dlogits") else 8 if k in INT64 else 4
        assert call(red, name, t, **{k: v + need // 2}) == RED_ERR_ALIGN, k
    # a null pointer is reported before an alignment
    k = REQUIRED[name][1]
    assert call(red, name, t, **{k: None, "logits": A + 1}) == RED_ERR_INVALID


def test_python_checks(red):
    torch = pytest.importorskip("torch")
    z = torch.zeros(3, 5)
    y = torch.zeros(3, dtype=torch.long)
    v = torch.zeros(3)
    with pytest.raises(ValueError):  # host tensors
        red.token_logprob_f32(z, y, v, v)
    with pytest.raises(TypeError):  # another element type
        red.token_logprob_bf16(z, y, v, v)
    with pytest.raises(TypeError):
        red.token_logprob_f32([[1.0]], y, v, v)
    for name in CALLS:
        for t in SIZE:
            f = getattr(red, "%s_%s" % (name, t))
            assert f.__doc__ and f.__name__ == "%s_%s" % (name, t)
    assert ctypes.sizeof(ctypes.c_size_t) == 8


@pytest.mark.parametrize("name,t", PAIRS)
def test_python_arguments(red, name, t):
    """Names, order and defaults of the Python functions, and what a call with
    the wrong ones raises before any tensor is looked at."""
    import inspect

    f = getattr(red, "%s_%s" % (name, t))
    names = list(inspect.signature(f).parameters)
    assert names[0] == "logits" and names[-1] == "stream"
    need = [k for k, p in inspect.signature(f).parameters.items()
            if p.default is inspect.Parameter.empty]
    assert names[:len(need)] == need
    with pytest.raises(TypeError, match="missing"):
        f(*[None] * (len(need) - 1))
    with pytest.raises(TypeError, match="unexpected"):
        f(*[None] * len(need), nothing=1)
    with pytest.raises(TypeError, match="multiple"):
        f(*[None] * len(need), logits=None)
    with pytest.raises(TypeError, match="at most"):
        f(*[None] * (len(names) + 1))
    with pytest.raises(TypeError, match="logits must be a torch.Tensor"):
        f(*[None] * len(need))
    with pytest.raises(TypeError, match="logits must be"):
        red.plan("%s_%s" % (name, t), *[None] * len(need))
