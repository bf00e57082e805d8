"""fp32_reductions_amd -- Python binding of libreduce (gfx950 HIP kernels).

Thin ctypes layer over the C ABI in ``include/reduce.h``: it checks that
torch tensors have the dtype, device and extent an entry point expects,
passes their device pointers and the current HIP stream, and turns a
non-zero status into ``ReduceError``.  Every step of the reduction runs in
the HIP kernels of ``libreduce.so``; there is no CPU fallback.  Importing
this package raises if the library has not been built
(``python fp32_reductions_amd/build.py``).

Names follow the C ABI:

    sum_f32 / max_f32 / min_f32 (x, out, accum=False, stream=None)
    sum_max_min_f32 (x, out[3], accum=False, stream=None)
    sum_f32_atomic / max_f32_atomic / min_f32_atomic (same)
    sum_rows_f32 / max_rows_f32 / min_rows_f32 (x, out, n=None, accum=False)
    sum_cols_f32 / max_cols_f32 / min_cols_f32 (src, out, C=None, accum=False)
    colprod_f32 / colprod_f16 / colprod_bf16 / colprod_i32 (src, out, C=None)
    colprod_i16 / colprod_u16 / colprod_u32 (src, out, C=None)

and, for _f32, _f16 and _bf16 logits, the losses over rows of logits

    token_logprob_f32 (logits, targets, logp, lse, ...)
    token_logprob_grad_f32 (logits, targets, lse, glogp, dlogits, ...)
    distill_topk_f32 (logits, idx, val, loss, ...)
    policy_loss_f32 (logits, targets, old_logp, advantage, loss, logp, ...)
    preference_loss_f32 (logits, targets, starts, loss, seq_logp, ...)

``plan(name, *args, **kwargs)`` marshals the same arguments once and returns
a ``Plan``; calling it enqueues the C entry point with the stored pointers,
sizes and stream, without re-checking the tensors.  The caller keeps the
tensors alive and unchanged in shape while the plan is in use.
"""
from __future__ import annotations

import ctypes
import inspect
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_PKG, "libreduce.so")

RED_OK, RED_ERR_INVALID, RED_ERR_ALIGN, RED_ERR_NOMEM, RED_ERR_HIP, RED_ERR_SCRATCH = range(6)


class ReduceError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_str(status), status))


if not os.path.exists(LIBRARY):
    raise ImportError(
        "libreduce.so is not built at %s; run "
        "'python fp32_reductions_amd/build.py' (hipcc, gfx950)" % LIBRARY)

_lib = ctypes.CDLL(LIBRARY)

_P, _SZ, _I, _F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
_SIGS = {
    "red_sum_f32": [_P, _SZ, _P, _I, _P],
    "red_max_f32": [_P, _SZ, _P, _I, _P],
    "red_min_f32": [_P, _SZ, _P, _I, _P],
    "red_sum_max_min_f32": [_P, _SZ, _P, _I, _P],
    "red_sum_max_min_f32_noalloc": [_P, _SZ, _P, _I, _P],
    "red_sum_f32_atomic": [_P, _SZ, _P, _I, _P],
    "red_max_f32_atomic": [_P, _SZ, _P, _I, _P],
    "red_min_f32_atomic": [_P, _SZ, _P, _I, _P],
    "red_sum_rows_f32": [_P, _SZ, _SZ, _SZ, _P, _I, _P],
    "red_max_rows_f32": [_P, _SZ, _SZ, _SZ, _P, _I, _P],
    "red_min_rows_f32": [_P, _SZ, _SZ, _SZ, _P, _I, _P],
    "red_sum_cols_f32": [_P, _SZ, _SZ, _SZ, _P, _I, _P],
    "red_max_cols_f32": [_P, _SZ, _SZ, _SZ, _P, _I, _P],
    "red_min_cols_f32": [_P, _SZ, _SZ, _SZ, _P, _I, _P],
    "red_colprod_f32": [_P, _SZ, _SZ, _SZ, _P, _P],
    "red_colprod_f16": [_P, _SZ, _SZ, _SZ, _P, _P],
    "red_colprod_bf16": [_P, _SZ, _SZ, _SZ, _P, _P],
    "red_colprod_i32": [_P, _SZ, _SZ, _SZ, _P, _P],
    "red_colprod_i16": [_P, _SZ, _SZ, _SZ, _P, _P],
    "red_colprod_u16": [_P, _SZ, _SZ, _SZ, _P, _P],
    "red_colprod_u32": [_P, _SZ, _SZ, _SZ, _P, _P],
    "red_release_workspace": [_P],
}
for _t in ("f32", "f16", "bf16"):
    _SIGS.update({
        "red_token_logprob_" + _t: [_P, _SZ, _SZ, _SZ, _P, _F, _P, _P, _P, _P],
        "red_token_logprob_grad_" + _t: [_P, _SZ, _SZ, _SZ, _P, _F, _P, _P, _P, _P, _P, _SZ, _P],
        "red_distill_topk_" + _t: [_P, _SZ, _SZ, _SZ, _P, _P, _SZ, _SZ, _P, _P, _F, _P, _I, _P,
                                   _P, _SZ, _P],
        "red_policy_loss_" + _t: [_P, _SZ, _SZ, _SZ, _P, _P, _P, _P, _P, _F, _F, _F, _F, _F, _P,
                                  _I, _P, _P, _P, _SZ, _P],
        "red_preference_loss_" + _t: [_P, _SZ, _SZ, _SZ, _P, _P, _SZ, _P, _P, _I, _F, _F, _F, _I,
                                      _P, _I, _P, _P, _SZ, _P],
    })
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _I
_lib.red_status_str.argtypes = [_I]
_lib.red_status_str.restype = ctypes.c_char_p
_lib.red_abi_version.argtypes = []
_lib.red_abi_version.restype = _I

EXPORTS = tuple(_SIGS) + ("red_status_str", "red_abi_version")


def lib() -> ctypes.CDLL:
    """The loaded libreduce (raw C ABI, for callers holding raw pointers)."""
    return _lib


def status_str(status: int) -> str:
    return _lib.red_status_str(status).decode()


def abi_version() -> int:
    return _lib.red_abi_version()


# The current stream's handle without a Stream object around it (2.5 us less
# per call), where this torch has the two functions.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
if _current_device is None:
    _raw_stream = None


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def release_workspace(stream=None) -> None:
    """Free the library's workspace for `stream` (the current stream when
    None) after the work enqueued on it has finished."""
    _check(_lib.red_release_workspace(_stream(stream)), "red_release_workspace")


def _check(status: int, where: str) -> None:
    if status != RED_OK:
        raise ReduceError(status, where)


class Plan:
    """A C entry point with its arguments already marshalled."""

    __slots__ = ("name", "fn", "args", "keep")

    def __init__(self, name, args, keep):
        self.name = name
        self.fn = getattr(_lib, name)
        self.args = args
        self.keep = keep  # the tensors whose pointers are in args

    def __call__(self) -> None:
        status = self.fn(*self.args)
        if status != RED_OK:
            raise ReduceError(status, self.name)


def _need(t: torch.Tensor, dtype, what: str) -> None:
    """dtype may be one torch dtype or a tuple of accepted dtypes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    ok = t.dtype in dtype if isinstance(dtype, tuple) else t.dtype == dtype
    if not ok:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.device.type != "cuda":
        raise ValueError("%s must be a device (cuda/HIP) tensor" % what)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)


# ---------------------------------------------------------------------------
# 1-D vector -> scalar
# ---------------------------------------------------------------------------

def _args_reduce1d(name: str, x, out, accum=False, stream=None):
    _need(x, torch.float32, "x")
    _need(out, torch.float32, "out")
    need = 3 if name.startswith("red_sum_max_min_f32") else 1
    if out.numel() < need:
        raise ValueError("out needs %d element(s)" % need)
    return (x.data_ptr(), x.numel(), out.data_ptr(), int(bool(accum)),
            _stream(stream)), (x, out)


def _reduce1d(name: str, x, out, accum, stream):
    args, _ = _args_reduce1d(name, x, out, accum, stream)
    _check(getattr(_lib, name)(*args), name)
    return out


def sum_f32(x, out, accum=False, stream=None):
    """out[0] = [out[0] +] sum(x), x any contiguous fp32 device tensor."""
    return _reduce1d("red_sum_f32", x, out, accum, stream)


def max_f32(x, out, accum=False, stream=None):
    return _reduce1d("red_max_f32", x, out, accum, stream)


def min_f32(x, out, accum=False, stream=None):
    return _reduce1d("red_min_f32", x, out, accum, stream)


def sum_max_min_f32(x, out, accum=False, stream=None):
    """out[0:3] = [out[0:3] (+, max, min)] (sum, max, min) of x, one read."""
    return _reduce1d("red_sum_max_min_f32", x, out, accum, stream)


def sum_max_min_f32_noalloc(x, out, accum=False, stream=None):
    """sum_max_min_f32 with its partials in the library's static scratch
    (no allocation); calls overlapping on one GPU race."""
    return _reduce1d("red_sum_max_min_f32_noalloc", x, out, accum, stream)


def sum_f32_atomic(x, out, accum=False, stream=None):
    return _reduce1d("red_sum_f32_atomic", x, out, accum, stream)


def max_f32_atomic(x, out, accum=False, stream=None):
    return _reduce1d("red_max_f32_atomic", x, out, accum, stream)


def min_f32_atomic(x, out, accum=False, stream=None):
    return _reduce1d("red_min_f32_atomic", x, out, accum, stream)


# ---------------------------------------------------------------------------
# segmented rows
# ---------------------------------------------------------------------------

def _args_rows(name: str, x, out, n=None, accum=False, stream=None):
    _need(x, torch.float32, "x")
    _need(out, torch.float32, "out")
    if x.dim() != 2:
        raise ValueError("x must be 2-D (rows, ld)")
    rows, ld = x.shape
    n = ld if n is None else int(n)
    if not 0 <= n <= ld:
        raise ValueError("need 0 <= n <= ld")
    if out.numel() < rows:
        raise ValueError("out needs one element per row")
    return (x.data_ptr(), rows, n, ld, out.data_ptr(), int(bool(accum)),
            _stream(stream)), (x, out)


def _rows(name: str, x, out, n, accum, stream):
    args, _ = _args_rows(name, x, out, n, accum, stream)
    _check(getattr(_lib, name)(*args), name)
    return out


def sum_rows_f32(x, out, n=None, accum=False, stream=None):
    """out[r] = [out[r] +] sum(x[r, :n]) for a row-major (rows, ld) x."""
    return _rows("red_sum_rows_f32", x, out, n, accum, stream)


def max_rows_f32(x, out, n=None, accum=False, stream=None):
    return _rows("red_max_rows_f32", x, out, n, accum, stream)


def min_rows_f32(x, out, n=None, accum=False, stream=None):
    return _rows("red_min_rows_f32", x, out, n, accum, stream)


# ---------------------------------------------------------------------------
# column sum / max / min
# ---------------------------------------------------------------------------

def _args_cols(name: str, src, out, C=None, accum=False, stream=None):
    _need(src, torch.float32, "src")
    _need(out, torch.float32, "out")
    if src.dim() != 2:
        raise ValueError("src must be 2-D (R, ld)")
    R, ld = src.shape
    C = ld if C is None else int(C)
    if not 0 <= C <= ld:
        raise ValueError("need 0 <= C <= ld")
    if out.numel() < C:
        raise ValueError("out needs C elements")
    return (src.data_ptr(), R, C, ld, out.data_ptr(), int(bool(accum)),
            _stream(stream)), (src, out)


def _cols(name: str, src, out, C, accum, stream):
    args, _ = _args_cols(name, src, out, C, accum, stream)
    _check(getattr(_lib, name)(*args), name)
    return out


def sum_cols_f32(src, out, C=None, accum=False, stream=None):
    """out[j] = [out[j] +] sum_i src[i, j] for j < C, fp32 (R, ld) tile."""
    return _cols("red_sum_cols_f32", src, out, C, accum, stream)


def max_cols_f32(src, out, C=None, accum=False, stream=None):
    return _cols("red_max_cols_f32", src, out, C, accum, stream)


def min_cols_f32(src, out, C=None, accum=False, stream=None):
    return _cols("red_min_cols_f32", src, out, C, accum, stream)


# ---------------------------------------------------------------------------
# column product
# ---------------------------------------------------------------------------

# Unsigned types may also arrive as the signed torch dtype of the same width
# (bit patterns): torch's uint16 / uint32 support on the device is partial.
_U16 = (torch.uint16, torch.int16) if hasattr(torch, "uint16") else (torch.int16,)
_U32 = (torch.uint32, torch.int32) if hasattr(torch, "uint32") else (torch.int32,)
_COLPROD_DTYPE = {"red_colprod_f32": torch.float32, "red_colprod_f16": torch.float16,
                  "red_colprod_bf16": torch.bfloat16, "red_colprod_i32": torch.int32,
                  "red_colprod_i16": torch.int16, "red_colprod_u16": _U16,
                  "red_colprod_u32": _U32}


def _args_colprod(name: str, src, out, C=None, stream=None):
    dtype = _COLPROD_DTYPE[name]
    _need(src, dtype, "src")
    _need(out, dtype, "out")
    if src.dim() != 2:
        raise ValueError("src must be 2-D (R, ld)")
    R, ld = src.shape
    C = ld if C is None else int(C)
    if not 0 <= C <= ld:
        raise ValueError("need 0 <= C <= ld")
    if out.numel() < C:
        raise ValueError("out needs C elements")
    return (src.data_ptr(), R, C, ld, out.data_ptr(), _stream(stream)), (src, out)


def _colprod(name: str, src, out, C, stream):
    args, _ = _args_colprod(name, src, out, C, stream)
    _check(getattr(_lib, name)(*args), name)
    return out


def colprod_f32(src, out, C=None, stream=None):
    """out[j] = prod_i src[i, j] for j < C (TCOLPROD), fp32."""
    return _colprod("red_colprod_f32", src, out, C, stream)


def colprod_f16(src, out, C=None, stream=None):
    """binary16 tile (torch.float16); fp32 products rounded once to fp16."""
    return _colprod("red_colprod_f16", src, out, C, stream)


def colprod_bf16(src, out, C=None, stream=None):
    """bfloat16 tile (torch.bfloat16); fp32 products rounded once to bf16."""
    return _colprod("red_colprod_bf16", src, out, C, stream)


def colprod_i32(src, out, C=None, stream=None):
    """int32 tile; products modulo 2^32."""
    return _colprod("red_colprod_i32", src, out, C, stream)


def colprod_i16(src, out, C=None, stream=None):
    """int16 tile; products modulo 2^16."""
    return _colprod("red_colprod_i16", src, out, C, stream)


def colprod_u16(src, out, C=None, stream=None):
    """uint16 tile (torch.uint16, or torch.int16 holding the bits); mod 2^16."""
    return _colprod("red_colprod_u16", src, out, C, stream)


def colprod_u32(src, out, C=None, stream=None):
    """uint32 tile (torch.uint32, or torch.int32 holding the bits); mod 2^32."""
    return _colprod("red_colprod_u32", src, out, C, stream)


# ---------------------------------------------------------------------------
# losses over rows of logits
# ---------------------------------------------------------------------------

_LOGITS_DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}


def _matrix(t, dtype, what: str):
    """(pointer, rows, columns, row stride) of a 2-D device tensor whose rows
    are contiguous; the row stride may exceed the columns."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a device (cuda/HIP) tensor" % what)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % what)
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("the rows of %s must be contiguous" % what)
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError("the rows of %s must not overlap" % what)
    return t.data_ptr(), rows, cols, ld


def _vector(t, dtype, n: int, what: str, optional: bool = False):
    """Pointer of a contiguous device tensor of exactly n elements (None: 0)."""
    if t is None and optional:
        return None
    _need(t, dtype, what)
    if t.numel() != n:
        raise ValueError("%s must have %d element(s), has %d" % (what, n, t.numel()))
    return t.data_ptr()


def _gradient(dlogits, dtype, rows: int, cols: int, optional: bool = True):
    if dlogits is None and optional:
        return None, 0
    ptr, r, c, ldd = _matrix(dlogits, dtype, "dlogits")
    if (r, c) != (rows, cols):
        raise ValueError("dlogits must have the shape of logits")
    return ptr, ldd


def _same_device(logits, *others) -> None:
    for t in others:
        if t is not None and t.device != logits.device:
            raise ValueError("all tensors must be on the device of logits")


def _args_token_logprob(name, logits, targets, logp, lse, entropy=None, scale=1.0, stream=None):
    """logp[r] = ln p_target, lse[r] = ln sum exp(scale * logits[r]) and, where
    given, entropy[r] of each row's softmax p at inverse temperature `scale`.

    logits (rows, V) with contiguous rows of any stride; targets int64 (a
    target outside [0, V) gives logp 0); logp, lse, entropy fp32."""
    dtype = _LOGITS_DTYPE[name.rsplit("_", 1)[1]]
    z, rows, V, ld = _matrix(logits, dtype, "logits")
    f32 = torch.float32
    _same_device(logits, targets, logp, lse, entropy)
    return (z, rows, V, ld, _vector(targets, torch.int64, rows, "targets"), float(scale),
            _vector(logp, f32, rows, "logp"), _vector(lse, f32, rows, "lse"),
            _vector(entropy, f32, rows, "entropy", True),
            _stream(stream)), (logits, targets, logp, lse, entropy)


def _args_token_logprob_grad(name, logits, targets, lse, glogp, dlogits, entropy=None,
                             gentropy=None, scale=1.0, stream=None):
    """dlogits from the gradients glogp (of logp) and gentropy (of entropy) of
    token_logprob, whose lse and entropy the caller kept.  dlogits may be
    logits itself."""
    dtype = _LOGITS_DTYPE[name.rsplit("_", 1)[1]]
    z, rows, V, ld = _matrix(logits, dtype, "logits")
    f32 = torch.float32
    dz, ldd = _gradient(dlogits, dtype, rows, V, False)
    if gentropy is not None and entropy is None:
        raise ValueError("gentropy needs entropy")
    _same_device(logits, targets, lse, glogp, dlogits, entropy, gentropy)
    return (z, rows, V, ld, _vector(targets, torch.int64, rows, "targets"), float(scale),
            _vector(lse, f32, rows, "lse"), _vector(entropy, f32, rows, "entropy", True),
            _vector(glogp, f32, rows, "glogp"), _vector(gentropy, f32, rows, "gentropy", True),
            dz, ldd, _stream(stream)), (logits, targets, lse, glogp, dlogits, entropy, gentropy)


def _args_distill_topk(name, logits, idx, val, loss, dlogits=None, teacher_lse=None, weight=None,
                       row_loss=None, scale=1.0, accum=False, stream=None):
    """loss[0] = [loss[0] +] sum_r weight[r] KL(teacher || softmax(scale *
    logits[r])) for a teacher given by K columns idx (rows, K) int64 and
    their logits val (rows, K) fp32; columns outside [0, V) are padding.
    Without teacher_lse the teacher is the softmax of its entries; with the
    log-sum-exp of its whole scaled row, the columns not listed count as one
    more.  weight: 1 / rows each when None; 0 leaves a row out.  dlogits
    takes the gradient (it may be logits itself), row_loss the rows' losses."""
    dtype = _LOGITS_DTYPE[name.rsplit("_", 1)[1]]
    z, rows, V, ld = _matrix(logits, dtype, "logits")
    f32 = torch.float32
    i, irows, K, ldk = _matrix(idx, torch.int64, "idx")
    v, vrows, vk, ldv = _matrix(val, f32, "val")
    if irows != rows or vrows != rows or vk != K:
        raise ValueError("idx and val must both be (rows, K)")
    if ldk != ldv:
        raise ValueError("idx and val must have the same row stride")
    dz, ldd = _gradient(dlogits, dtype, rows, V)
    _same_device(logits, idx, val, loss, dlogits, teacher_lse, weight, row_loss)
    return (z, rows, V, ld, i, v, K, ldk, _vector(teacher_lse, f32, rows, "teacher_lse", True),
            _vector(weight, f32, rows, "weight", True), float(scale),
            _vector(loss, f32, 1, "loss"), int(bool(accum)),
            _vector(row_loss, f32, rows, "row_loss", True), dz, ldd,
            _stream(stream)), (logits, idx, val, loss, dlogits, teacher_lse, weight, row_loss)


def _args_policy_loss(name, logits, targets, old_logp, advantage, loss, logp, dlogits=None,
                      ref_logp=None, weight=None, entropy=None, scale=1.0, clip_low=0.2,
                      clip_high=0.2, kl_coef=0.0, entropy_coef=0.0, accum=False, stream=None):
    """loss[0] = [loss[0] +] sum_r weight[r] (-min(ratio A, clip(ratio) A) +
    kl_coef (exp(d) - d - 1) - entropy_coef H) with ratio = exp(logp[r] -
    old_logp[r]) clipped to [1 - clip_low, 1 + clip_high], A = advantage[r],
    d = ref_logp[r] - logp[r] and H the entropy of softmax(scale *
    logits[r]).  logp and entropy take the rows' values, dlogits the gradient
    (it may be logits itself).  weight: 1 / rows each when None; rows of
    weight 0, or without a target in [0, V), do not count."""
    dtype = _LOGITS_DTYPE[name.rsplit("_", 1)[1]]
    z, rows, V, ld = _matrix(logits, dtype, "logits")
    f32 = torch.float32
    dz, ldd = _gradient(dlogits, dtype, rows, V)
    if kl_coef and ref_logp is None:
        raise ValueError("kl_coef needs ref_logp")
    _same_device(logits, targets, old_logp, advantage, loss, logp, dlogits, ref_logp, weight,
                 entropy)
    return (z, rows, V, ld, _vector(targets, torch.int64, rows, "targets"),
            _vector(old_logp, f32, rows, "old_logp"),
            _vector(ref_logp, f32, rows, "ref_logp", True),
            _vector(advantage, f32, rows, "advantage"),
            _vector(weight, f32, rows, "weight", True), float(scale), float(clip_low),
            float(clip_high), float(kl_coef), float(entropy_coef),
            _vector(loss, f32, 1, "loss"), int(bool(accum)), _vector(logp, f32, rows, "logp"),
            _vector(entropy, f32, rows, "entropy", True), dz, ldd,
            _stream(stream)), (logits, targets, old_logp, advantage, loss, logp, dlogits,
                               ref_logp, weight, entropy)


def _args_preference_loss(name, logits, targets, starts, loss, seq_logp, dlogits=None,
                          ref_logp=None, weight=None, kind="sigmoid", beta=0.1, margin=0.0,
                          smoothing=0.0, average=False, accum=False, stream=None):
    """loss[0] = [loss[0] +] sum_p weight[p] l(beta D_p - margin), D_p the
    log-ratio of pair p's chosen sequence (number p) over its rejected one
    (number pairs + p), each against ref_logp; l is "sigmoid" (with label
    smoothing), "hinge" or "squared".  Sequence i has the rows starts[i] to
    starts[i + 1] (int64, 2 * pairs + 1 of them); seq_logp (2 * pairs) takes
    the sums (average: means) of their targets' log-probabilities, dlogits the
    gradient (it may be logits itself).  weight: 1 / pairs each when None."""
    dtype = _LOGITS_DTYPE[name.rsplit("_", 1)[1]]
    z, rows, V, ld = _matrix(logits, dtype, "logits")
    f32 = torch.float32
    _need(starts, torch.int64, "starts")
    if starts.numel() % 2 == 0:
        raise ValueError("starts must have 2 * pairs + 1 elements")
    pairs = starts.numel() // 2
    if kind not in PREFERENCE_KINDS:
        raise ValueError("kind must be one of %s" % ", ".join(sorted(PREFERENCE_KINDS)))
    dz, ldd = _gradient(dlogits, dtype, rows, V)
    _same_device(logits, targets, starts, loss, seq_logp, dlogits, ref_logp, weight)
    return (z, rows, V, ld, _vector(targets, torch.int64, rows, "targets"), starts.data_ptr(),
            pairs, _vector(ref_logp, f32, 2 * pairs, "ref_logp", True),
            _vector(weight, f32, pairs, "weight", True), PREFERENCE_KINDS[kind], float(beta),
            float(margin), float(smoothing), int(bool(average)), _vector(loss, f32, 1, "loss"),
            int(bool(accum)), _vector(seq_logp, f32, 2 * pairs, "seq_logp"), dz, ldd,
            _stream(stream)), (logits, targets, starts, loss, seq_logp, dlogits, ref_logp, weight)


_ROWLOSS = {"token_logprob": _args_token_logprob, "token_logprob_grad": _args_token_logprob_grad,
            "distill_topk": _args_distill_topk, "policy_loss": _args_policy_loss,
            "preference_loss": _args_preference_loss}


def _typed(cname: str, marshal):
    """The public function of one C entry point: marshal, call, check."""
    fn = getattr(_lib, cname)

    def call(*args, **kwargs):
        cargs, _ = marshal(cname, *args, **kwargs)
        _check(fn(*cargs), cname)

    sig = inspect.signature(marshal)
    call.__signature__ = sig.replace(parameters=list(sig.parameters.values())[1:])
    call.__name__ = call.__qualname__ = cname[len("red_"):]
    call.__doc__ = marshal.__doc__
    return call


for _name, _marshal in _ROWLOSS.items():
    for _t in _LOGITS_DTYPE:
        globals()["%s_%s" % (_name, _t)] = _typed("red_%s_%s" % (_name, _t), _marshal)


# ---------------------------------------------------------------------------
# pre-marshalled calls
# ---------------------------------------------------------------------------

_MARSHAL = {}
for _op in ("sum", "max", "min"):
    _MARSHAL["%s_f32" % _op] = ("red_%s_f32" % _op, _args_reduce1d)
    _MARSHAL["%s_f32_atomic" % _op] = ("red_%s_f32_atomic" % _op, _args_reduce1d)
    _MARSHAL["%s_rows_f32" % _op] = ("red_%s_rows_f32" % _op, _args_rows)
    _MARSHAL["%s_cols_f32" % _op] = ("red_%s_cols_f32" % _op, _args_cols)
_MARSHAL["sum_max_min_f32"] = ("red_sum_max_min_f32", _args_reduce1d)
_MARSHAL["sum_max_min_f32_noalloc"] = ("red_sum_max_min_f32_noalloc", _args_reduce1d)
for _t in ("f32", "f16", "bf16", "i32", "i16", "u16", "u32"):
    _MARSHAL["colprod_" + _t] = ("red_colprod_" + _t, _args_colprod)
for _name, _marshal in _ROWLOSS.items():
    for _t in _LOGITS_DTYPE:
        _MARSHAL["%s_%s" % (_name, _t)] = ("red_%s_%s" % (_name, _t), _marshal)


def plan(name: str, *args, **kwargs) -> Plan:
    """Marshal the arguments of entry point ``name`` (e.g. "sum_f32") once;
    the returned Plan enqueues the call each time it is called."""
    cname, marshal = _MARSHAL[name]
    cargs, keep = marshal(cname, *args, **kwargs)
    return Plan(cname, cargs, keep)
