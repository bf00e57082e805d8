"""The losses over rows of logits in fp64, written from their definitions in
include/reduce.h, with the error each kernel may make.

Everything takes CPU tensors.  Every function returns values and bounds side
by side; the bounds follow from u = 2^-24 (half an fp32 step) and, for results
of type T, half a step of T:

* a term 2^((z - m) c) of a row's sum: its exponent x ln 2 = scale (z - m) is
  rounded in c and in the fused product (2 |x| u), v_exp_f32 is good to a step
  (2 u), so the term is off by (2 |x| + 2) u of itself.  Averaged over the row
  with weights p the |x| come to at most ln V + 1.
* the sum: a thread adds at most V / 1024 (rows shared by 256 threads and
  more; 64 in shorter ones' four accumulators: 16) terms one after another,
  and 24 more additions and moves to a new maximum (4 u each) join threads and
  waves: (V / 1024 + 16 + 4 * 24) u.
Together S, and so ln S, is off by stat_error(V) below.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24


def stat_error(V: int) -> float:
    return U * (2 * math.log(V) + 4 + V / 1024 + 16 + 4 * 24)


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def floor_of(dtype) -> float:
    """Half the smallest step of the type, and the terms below 2^-126 of the
    largest that count as zero."""
    info = torch.finfo(dtype)
    return max(info.tiny * info.eps / 2, 2.0 ** -125)


class Rows:
    """Softmax statistics of the rows of z at inverse temperature `scale`."""

    def __init__(self, z, scale):
        self.z = z.double()
        self.scale = float(torch.tensor(scale, dtype=torch.float32))
        x = self.z * self.scale
        self.V = z.shape[1]
        m = x.amax(1, keepdim=True)
        ref = torch.where(m == -math.inf, torch.zeros_like(m), m)
        e = (x - ref).exp()
        s = e.sum(1, keepdim=True)
        self.lse = (ref + s.log()).squeeze(1)
        self.lnp = x - ref - s.log()
        self.p = e / s
        self.minus_lnp = torch.where(self.p > 0, -self.lnp, torch.zeros_like(self.lnp))
        self.entropy = (self.p * self.minus_lnp).sum(1)
        bad = s.squeeze(1)
        self.entropy = torch.where((bad > 0) & (bad < math.inf), self.entropy,
                                   torch.full_like(self.entropy, math.nan))
        self.err = stat_error(self.V)
        # an entropy is a mean of |ln p|: each factor's error times the other
        self.entropy_err = self.err * 3 * (math.log(self.V) + 1) + self.entropy.abs() * U

    def p_err(self):
        return self.p * (self.err + U * (2 * self.minus_lnp + 4))


def hits(targets, V):
    ok = (targets >= 0) & (targets < V)
    return ok, torch.where(ok, targets, torch.zeros_like(targets))


def onehot(r: Rows, targets):
    ok, y = hits(targets, r.V)
    d = torch.zeros_like(r.p)
    d.scatter_(1, y.unsqueeze(1), ok.double().unsqueeze(1))
    return d


def token_logprob(z, targets, scale):
    """{name: (value, bound)}"""
    r = Rows(z, scale)
    ok, y = hits(targets, r.V)
    logp = torch.where(ok, r.lnp.gather(1, y.unsqueeze(1)).squeeze(1),
                       torch.zeros(len(y), dtype=torch.double))
    return {"logp": (logp, r.err + logp.abs() * U), "lse": (r.lse, r.err + r.lse.abs() * U),
            "entropy": (r.entropy, r.entropy_err)}


def round_bound(value, dtype):
    return value.abs() * half_step(dtype) * 1.001 + floor_of(dtype)


def token_logprob_grad(z, targets, scale, lse, glogp, gentropy=None, entropy=None):
    """The definition takes lse and entropy as they are handed over."""
    r = Rows(z, scale)
    ok, _ = hits(targets, r.V)
    g = torch.where(ok, glogp.double(), torch.zeros(len(glogp), dtype=torch.double)).unsqueeze(1)
    lnp = r.z * r.scale - lse.double().unsqueeze(1)
    p = lnp.exp()
    lnp = torch.where(p > 0, lnp, torch.zeros_like(lnp))
    d = g * (onehot(r, targets) - p)
    # exponent: two roundings of |ln p|, and of the shift's remainder; then
    # a few operations on the product
    rel = U * (4 * lnp.abs() + 16)
    err = g.abs() * (p * rel + onehot(r, targets) * 2 * U)
    if gentropy is not None:
        h, H = gentropy.double().unsqueeze(1), entropy.double().unsqueeze(1)
        d = d - h * p * (lnp + H)
        err = err + h.abs() * p * (lnp.abs() + H.abs()) * (rel + 8 * U)
    live = (g != 0) | ((gentropy.double().unsqueeze(1) != 0) if gentropy is not None else False)
    d = torch.where(live, d * r.scale, torch.zeros_like(d))
    err = torch.where(live, err * r.scale, torch.zeros_like(err))
    return d, err + round_bound(d, z.dtype)


def _zero_dead(live, *values):
    out = []
    for v in values:
        m = live if v.dim() == 1 else live.unsqueeze(1)
        out.append(torch.where(m, v, torch.zeros_like(v)))
    return out


def total(row, err, weight):
    """Weighted sum of row losses and its bound."""
    w = weight.double()
    live = w != 0
    s = torch.where(live, row * w, torch.zeros_like(row)).sum()
    e = torch.where(live, (err + row.abs() * 2.0 ** -50) * w.abs(), torch.zeros_like(row)).sum()
    return s, e + s.abs() * U + 1e-40


def distill_topk(z, idx, val, scale, weight, teacher_lse=None):
    """Loss, row losses and gradient, each (value, bound)."""
    r = Rows(z, scale)
    rows, V = z.shape
    listed = (idx >= 0) & (idx < V)
    at = torch.where(listed, idx, torch.zeros_like(idx))
    t = torch.where(listed, val.double() * r.scale, torch.full(val.shape, -math.inf).double())
    live = weight != 0
    if teacher_lse is None:
        top = t.amax(1, keepdim=True)
        live = live & (top.squeeze(1) != -math.inf)
        ref = torch.where(top == -math.inf, torch.zeros_like(top), top)
        lnq = t - ref - (t - ref).exp().sum(1, keepdim=True).log()
    else:
        lnq = t - teacher_lse.double().unsqueeze(1)
    q = torch.where(listed, lnq.exp(), torch.zeros_like(t))
    lnp_at = r.lnp.gather(1, at)
    row = torch.where(q != 0, q * (lnq - lnp_at), torch.zeros_like(q)).sum(1)
    Q = q.sum(1)
    row_err = Q * r.err
    # q per column (entries of one column add up)
    inside = torch.zeros(rows, V, dtype=torch.bool)
    qv = torch.zeros(rows, V, dtype=torch.double)
    for i in range(rows):
        for k in range(idx.shape[1]):
            if listed[i, k]:
                inside[i, at[i, k]] = True
                qv[i, at[i, k]] += q[i, k]
    mass = Q.clone()
    d_out = torch.zeros(rows, 1, dtype=torch.double)
    if teacher_lse is not None:
        rest = torch.where((inside.sum(1) < V) & (Q < 1), 1 - Q, torch.zeros_like(Q))
        left = torch.where(inside, torch.zeros_like(r.p), r.p).sum(1)
        # ln p_r from the terms outside alone, which stay exact when tiny
        ln_left = torch.where(inside, torch.full_like(r.lnp, -math.inf), r.lnp).logsumexp(1)
        row = row + torch.where(rest > 0, rest * (rest.clamp_min(1e-300).log() - ln_left),
                                torch.zeros_like(rest))
        row_err = row_err + rest * 2 * r.err
        mass = Q + rest
        d_out = torch.where(left > 0, rest / left.clamp_min(1e-300), torch.zeros_like(rest))
        d_out = d_out.unsqueeze(1)
    mass = mass.unsqueeze(1)
    d = torch.where(inside, r.p * mass - qv, r.p * (mass - d_out))
    err = torch.where(inside, r.p_err() * mass + 2 * U * (r.p * mass + qv),
                      (r.p_err() + 2 * r.err * r.p) * (mass + d_out))
    f = (weight.double() * r.scale).unsqueeze(1)
    row_err = row_err + row.abs() * U
    row, row_err, d, err = _zero_dead(live, row, row_err, d * f, err * f.abs())
    err = err + d.abs() * 4 * U
    loss = total(row, row_err, torch.where(live, weight, torch.zeros_like(weight)))
    return {"loss": loss, "row_loss": (row, row_err), "dlogits": (d, err + round_bound(d, z.dtype))}


def policy_loss(z, targets, old_logp, advantage, weight, scale=1.0, ref_logp=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, entropy_coef=0.0):
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    clip_low, clip_high, kl_coef, entropy_coef = map(f32, (clip_low, clip_high, kl_coef,
                                                           entropy_coef))
    r = Rows(z, scale)
    ok, y = hits(targets, r.V)
    live = ok & (weight != 0)
    logp = r.lnp.gather(1, y.unsqueeze(1)).squeeze(1)
    adv = advantage.double()
    ratio = (logp - old_logp.double()).exp()
    free = ratio * adv
    clipped = ratio.clamp(1 - clip_low, 1 + clip_high) * adv
    cut = free > clipped
    row = torch.where(cut, -clipped, -free)
    g = torch.where(cut, torch.zeros_like(free), -free)
    slack = r.err  # of ln p
    row_err = free.abs() * slack * 2
    g_err = free.abs() * slack * 2
    if kl_coef != 0:
        k = ref_logp.double() - logp
        row = row + kl_coef * (torch.expm1(k) - k)
        row_err = row_err + abs(kl_coef) * torch.expm1(k).abs() * slack * 2
        g = g - kl_coef * torch.expm1(k)
        g_err = g_err + abs(kl_coef) * k.exp() * slack * 2
    H = r.entropy
    row = row - entropy_coef * H if entropy_coef else row
    row_err = row_err + abs(entropy_coef) * r.entropy_err
    hot = onehot(r, targets)
    G, GE = g.unsqueeze(1), g_err.unsqueeze(1)
    d = G * (hot - r.p)
    err = G.abs() * (r.p_err() + 4 * U * (hot + r.p)) + GE * (hot + r.p)
    if entropy_coef:
        lnp = -r.minus_lnp
        He = H.unsqueeze(1)
        d = d + entropy_coef * r.p * (lnp + He)
        err = err + abs(entropy_coef) * (
            r.p_err() * (lnp.abs() + He) + r.p * (U * (8 * lnp.abs() + 8 * He + 8) + 2 * r.err
                                                  + r.entropy_err.unsqueeze(1)))
    f = (weight.double() * r.scale).unsqueeze(1)
    logp_err, ent_err = r.err + logp.abs() * U, r.entropy_err
    logp, logp_err, H, ent_err, row, row_err, d, err = _zero_dead(
        live, logp, logp_err, H, ent_err, row, row_err, d * f, err * f.abs())
    loss = total(row, row_err, torch.where(live, weight, torch.zeros_like(weight)))
    return {"loss": loss, "logp": (logp, logp_err), "entropy": (H, ent_err),
            "dlogits": (d, err + d.abs() * 4 * U + round_bound(d, z.dtype))}


def preference_loss(z, targets, starts, weight, ref_logp=None, kind="sigmoid", beta=0.1,
                    margin=0.0, smoothing=0.0, average=False):
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    beta, margin, smoothing = map(f32, (beta, margin, smoothing))
    r = Rows(z, 1.0)
    rows = z.shape[0]
    ok, y = hits(targets, r.V)
    zero = torch.zeros(rows, dtype=torch.double)
    logp = torch.where(ok, r.lnp.gather(1, y.unsqueeze(1)).squeeze(1), zero)
    bound = starts.clamp(0, rows).tolist()
    n = len(bound) // 2
    seq, count, seq_err = [], [], []
    for a, b in zip(bound[:-1], bound[1:]):
        c = max(1, int(ok[a:b].sum())) if average else 1
        seq.append(logp[a:b].sum() / c)
        count.append(c)
        seq_err.append(float(ok[a:b].sum()) * r.err / c)
    seq, seq_err = torch.stack(seq), torch.tensor(seq_err, dtype=torch.double)
    ref = ref_logp.double() if ref_logp is not None else torch.zeros(2 * n, dtype=torch.double)
    delta = (seq - ref)[:n] - (seq - ref)[n:]
    delta_err = seq_err[:n] + seq_err[n:]
    h, h_err = beta * delta - margin, beta * delta_err
    if kind == "sigmoid":
        up, down = torch.sigmoid(h), torch.sigmoid(-h)
        sp = torch.nn.functional.softplus
        loss = (1 - smoothing) * sp(-h) + smoothing * sp(h)
        slope = smoothing * up - (1 - smoothing) * down
        steep = 0.25
    elif kind == "hinge":
        loss = (1 - h).clamp_min(0)
        slope = torch.where(h >= 1, torch.zeros_like(h), -torch.ones_like(h))
        steep = 0.0
    else:
        d = (h - 0.5) / beta
        loss, slope = d * d, 2 * d / beta
        steep = 2 / beta ** 2
    w = weight.double()
    live = w != 0
    g = torch.where(live, w * slope * beta, torch.zeros_like(w))
    g_err = torch.where(live, w.abs() * beta * steep * h_err, torch.zeros_like(w))
    sum_, err = total(loss, (slope.abs() + steep * h_err) * h_err, weight)
    row_g, row_ge = zero.clone(), zero.clone()
    for i, (a, b) in enumerate(zip(bound[:-1], bound[1:])):
        p = i % n
        row_g[a:b] = (g[p] if i < n else -g[p]) / count[i]
        row_ge[a:b] = g_err[p] / count[i]
    row_g, row_ge = torch.where(ok, row_g, zero), torch.where(ok, row_ge, zero)
    hot = onehot(r, targets)
    G = row_g.unsqueeze(1)
    d = G * (hot - r.p)
    derr = G.abs() * (r.p_err() + 4 * U * (hot + r.p)) + row_ge.unsqueeze(1) * (hot + r.p)
    d, derr = _zero_dead(row_g != 0, d, derr)
    return {"loss": (sum_, err), "seq_logp": (seq, seq_err + seq.abs() * U),
            "dlogits": (d, derr + d.abs() * 4 * U + round_bound(d, z.dtype))}


def check(name, got, value, bound):
    """got within bound of value; NaN and infinities where value has them."""
    got, value = got.double().cpu(), value.double().cpu()
    bound = torch.as_tensor(bound, dtype=torch.double).expand_as(value)
    fine = value.isfinite()
    same = (got == value) | (got.isnan() & value.isnan())
    bad = torch.where(fine, ~((got - value).abs() <= bound), ~same)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s%s: got %r, want %r within %g (%d of %d off)" % (
            name, list(i), got[i].item(), value[i].item(), bound[i].item(), int(bad.sum()),
            bad.numel()))
