"""The operators around the output layer in fp64, written from their definitions
in include/reduce.h, with the error each kernel may make.

Everything takes tensors of one device and returns {output: (value, bound)}.  u = 2^-24
is half an fp32 step; a result of type T adds half a step of T (half_step, and
below its normal range half the smallest step, floor_of).
"""
from __future__ import annotations

import math

import torch

from rowloss_reference import U, floor_of, half_step

E4M3 = torch.float8_e4m3fn


def f32(v: float) -> float:
    return float(torch.tensor(v, dtype=torch.float32))


def rounded(value, error, dtype):
    """`error` before the rounding to dtype, and the rounding."""
    h = half_step(dtype)
    return value, error * (1 + h) + value.abs() * h + floor_of(dtype)


def same(name, got, value, bound):
    """got within bound of value; NaN where value is NaN and only there."""
    got = got.detach().to(value.device).double()
    bound = torch.as_tensor(bound, dtype=torch.float64, device=value.device)
    assert got.shape == value.shape, (name, got.shape, value.shape)
    nan = value.isnan()
    assert torch.equal(got.isnan(), nan), (name, "NaN", got.isnan().sum(), nan.sum())
    inf = value.isinf()
    assert torch.equal(got[inf], value[inf]), (name, "infinities")
    fine = ~nan & ~inf
    off = (got - value).abs()[fine]
    bound = bound.expand_as(value)[fine]
    bad = ~(off <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %g at %g allowed" % (
        name, bad.sum(), bad.numel(), (off / bound)[bad].max() if bad.any() else 0,
        bound[bad].max())


def add_rmsnorm(x, residual, weight, eps):
    """x + residual is one fp32 step (u).  The sum of squares is fp64, and
    rstd's root and quotient are too, rounded once: rstd is off by what the
    h are (u each, at most u on average) and u, so 2 u.  y is two products
    more: 2 u + 2 u + u for h itself = 5 u."""
    dtype = x.dtype
    h = x.double() + (residual.double() if residual is not None else 0.0)
    r = (h.square().mean(1) + f32(eps)).rsqrt()
    y = h * r.unsqueeze(1) * weight.double()
    eh = U * h.abs() if residual is not None else torch.zeros_like(h)
    return {"sum": rounded(h, eh, dtype), "rstd": rounded(r, 2 * U * r, torch.float32),
            "y": rounded(y, 5 * U * y.abs(), dtype), "exact": y}


def check_8bit(y8, yscale, y):
    """The scale is the largest |y| (5 u off) over 448 (u); a value is off by
    half a step of its own, 2^-4 of itself or half the smallest step 2^-9 of the scale,
    and by the scale's and y's errors (5 u + 6 u + 2 u of itself, doubled where
    a tie falls the other way: those sit within the half step's own bound)."""
    most = y.abs().amax(1)
    same("yscale", yscale, most / 448.0, 7 * U * most / 448.0)
    q = y8.to(y.device).to(torch.float32).double()
    s = (most / 448.0).unsqueeze(1)
    step = torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10)
    off = (q * s - y).abs()
    assert (off <= step * (1 + 2.0 ** -10) + 16 * U * y.abs()).all(), (off / step).max()


def rmsnorm_grad(h, weight, rstd, dy, dsum):
    """n is one product (u), g another; the mean of g n is fp64 of fp32 factors
    (2 u of the sum of |g n|) rounded once; n rstd mean two products (3 u more),
    the difference one step and the product with rstd another, dsum one.  dw adds
    at most rows / groups terms, each two products (2 u), in fp32 one after
    another (a workgroup takes at most ceil(rows / 1) of them; 64 and 4 more
    where rows share a wave or workgroup), then fp64."""
    n = h.double() * rstd.double().unsqueeze(1)
    g = dy.double() * weight.double()
    D, rows = h.shape[1], h.shape[0]
    r = rstd.double().abs().unsqueeze(1)
    c = (g * n).mean(1, keepdim=True)
    ca = (g * n).abs().mean(1, keepdim=True)
    dx = (g - n * c) * rstd.double().unsqueeze(1)
    err = U * r * (3 * g.abs() + n.abs() * (6 * c.abs() + 3 * ca))
    if dsum is not None:
        dx = dx + dsum.double()
        err = err + U * dx.abs()
    t = dy.double() * n
    dw = t.sum(0)
    return {"dx": rounded(dx, err, h.dtype),
            "dweight": rounded(dw, U * t.abs().sum(0) * (2 + min(rows, 1024) + 8), torch.float32)}


def router_balance(z, experts, weight, balance, zc):
    """A softmax term's exponent is a difference and a product (2 |x| u) and
    v_exp_f32 a step (2 u); the row's sum at most 32 terms one after another and
    6 more; so p is off by (2 |x| + 2 ln E + 46) u of itself.  P adds rows in
    fp32, then 10 joins, then fp64."""
    rows, E = z.shape
    w = (torch.full((rows,), 1.0 / rows, device=z.device) if weight is None else weight).double()
    live = w != 0
    x = z.double()
    lse = x.logsumexp(1)
    p = (x - lse.unsqueeze(1)).exp()
    p = torch.where(live.unsqueeze(1), p, 0.0)
    lse = torch.where(live, lse, 0.0)
    e = experts[live].reshape(-1)
    counts = torch.bincount(e[(e >= 0) & (e < E)], minlength=E)
    total = int(counts.sum())
    f = counts.double() / max(1, total)
    P = (p * w.unsqueeze(1)).sum(0)
    b, c = f32(balance), f32(zc)
    loss = b * E * (f * P).sum() if total else torch.zeros_like(P.sum())
    loss = loss + c * (w * lse * lse).sum()
    q = b * E * f
    depth = torch.where(p > 0, (x - x.amax(1, keepdim=True)).abs(), 0.0)
    ep = (2 * depth + 2 * math.log(E) + 48) * U * p
    eP = (ep * w.abs().unsqueeze(1)).sum(0) + U * (p * w.abs().unsqueeze(1)).sum(0) * (rows + 16)
    inner = q - (p * q).sum(1, keepdim=True) + 2 * c * lse.unsqueeze(1)
    d = w.unsqueeze(1) * p * inner
    # the row's sum of p q (its terms' errors, 40 additions) and of lse: fp32
    ei = (ep * q.abs()).sum(1, keepdim=True) + 40 * U * (p * q.abs()).sum(1, keepdim=True)
    el = U * (4 * lse.abs() + 8 + 2 * math.log(E) + 48).unsqueeze(1)
    ei = ei + 2 * abs(c) * el + 6 * U * (q.abs() + (2 * c * lse).abs().unsqueeze(1))
    ed = w.abs().unsqueeze(1) * (ep * inner.abs() + p * ei) + 6 * U * d.abs()
    eloss = abs(b) * E * (f * eP).sum() + abs(c) * (
        w.abs() * (2 * lse.abs() * el.squeeze(1) + U * lse * lse)).sum()
    return {"counts": (counts.double(), 0.0),
            "prob": rounded(P, eP, torch.float32),
            "loss": rounded(loss.reshape(1), eloss.reshape(1), torch.float32),
            "dlogits": rounded(d, ed, z.dtype)}


def linear_ce(hidden, weight, targets, row_weight, scale, zc):
    """A product of 16-bit values is exact in fp32 and the sum of D of them, in
    any order of blocks, is off by at most D u sum |h w|: the matrix cores add
    16 at a time, so (D / 16 + 16) u bounds what they do (one rounding a block,
    and 16 within).  ez is that of a row's worst logit.  A term's exponent adds
    (|x| + 2) u, the row's sum V / tiles terms in fp32: 128 / 2 of a lane and 8
    joins, then fp64; so ln S is off by scale ez + stat.  d over its weight is rounded
    to the inputs' type before it is multiplied (half a step of each term; in f16,
    where it is 16 times larger, at least half of the smallest step, 2^-25 / 16 of the
    weight), and the sums over V and over rows are fp32: (V / 16 + 16) u, and as much
    for rows.  For dW the hidden rows carry their weights' exponents: exact, but for
    f16's smallest step, half of which is 2^-25 of up to twice the largest weight over
    the row's."""
    dtype = hidden.dtype
    rows, D = hidden.shape
    V = weight.shape[0]
    w = (torch.full((rows,), 1.0 / rows, device=hidden.device) if row_weight is None
         else row_weight).double()
    live = (w != 0) & (targets >= 0) & (targets < V)
    s, c = f32(scale), f32(zc)
    h = torch.where(live.unsqueeze(1), hidden.double(), 0.0)
    W = weight.double()
    z = h @ W.t()
    ez = ((D / 16 + 16) * U * (h.abs() @ W.abs().t())).amax(1)
    x = z * s
    lse = x.logsumexp(1)
    y = torch.where(live, targets, torch.zeros_like(targets))
    at = x.gather(1, y.unsqueeze(1)).squeeze(1)
    logp = torch.where(live, at - lse, 0.0)
    lse = torch.where(live, lse, 0.0)
    depth = (x.amax(1, keepdim=True) - x).clamp_max(100.0)
    p = torch.where(live.unsqueeze(1), (x - x.logsumexp(1, keepdim=True)).exp(), 0.0)
    # a term's relative error: two steps of its exponent, v_exp_f32, 80 additions
    stat = (2 * (p * depth).sum(1) + 2 + 80 + 4 * math.log(max(2, V))) * U
    el = s * ez + stat
    row = torch.where(live, c * lse * lse - logp, 0.0)
    loss = (w * row).sum().reshape(1)
    eloss = (w.abs() * (2 * el + abs(c) * 2 * lse.abs() * el)).sum().reshape(1)
    out = {"loss": rounded(loss, eloss, torch.float32),
           "logp": rounded(logp, torch.where(live, 2 * el, 0.0), torch.float32),
           "lse": rounded(lse, torch.where(live, el, 0.0), torch.float32)}
    a = (w * s * (1 + 2 * c * lse)).unsqueeze(1)
    b = torch.where(live, w * s, 0.0)
    d = a * p
    # of p: the logit's error, the lse's, its rounding times log2 e and the exponent's own
    ep = (s * ez + el + (4 * lse.abs() + 4) * U).unsqueeze(1) + 2 * depth * U
    ed = d.abs() * ep
    d = torch.where(live.unsqueeze(1), d, 0.0)
    d = d.scatter_add(1, y.unsqueeze(1), -b.unsqueeze(1))
    ed = ed + U * (a.abs() * p + d.abs()) * 4
    most = b.abs()
    small = 2.0 ** -25 / 16 * most.unsqueeze(1) if dtype == torch.float16 else 0.0
    ed = torch.where(live.unsqueeze(1), ed + half_step(dtype) * (d.abs() + ed) + small, 0.0)
    dh = d @ W
    edh = ed @ W.abs() + (V / 16 + 24) * U * (d.abs() @ W.abs())
    dw = d.t() @ h
    if dtype == torch.float16:  # the scaled copy of the hidden rows: its smallest steps
        lost = 2.0 ** -25 * 2 * most.max() * (d.abs() / most.clamp_min(1e-300).unsqueeze(1)).sum(0)
    edw = ed.t() @ h.abs() + (rows / 16 + 24) * U * (d.abs().t() @ h.abs())
    if dtype == torch.float16:
        edw = edw + lost.unsqueeze(1)
    out["dhidden"] = rounded(dh, edh, dtype)
    out["dweight"] = rounded(dw, edw, dtype)
    return out
