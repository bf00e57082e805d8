"""Measured cases of the losses over rows of logits.

Five operators read a row-major matrix of logits (one row for each token, V
columns) and reduce each row by its log-sum-exp:

    logprob     the log-probability of each row's target and the row's entropy
    grad        the gradient of those two with respect to the logits
    distill     the divergence from a teacher known by its K largest logits
    policy      the clipped ratio loss of a policy, with a KL term and entropy
    preference  the paired log-ratio loss of chosen and rejected sequences

Each case is one pass of one operator.  ``own`` selects the library's entry
points; otherwise the operators are computed by elementary torch operations
in fp32 (sums over many tokens in fp64), rounded once at the end.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_LARGEST = 1 << 30  # elements of the largest matrix of logits


def listed():
    return [
        # scoring one token while a sequence is generated: launch latency
        {"name": "logprob_one_token", "op": "logprob", "dtype": "bf16", "rows": 1, "V": 32768,
         "pad": 0, "entropy": False},
        # scoring a batch of sequences with the policy that wrote them
        {"name": "logprob_batch", "op": "logprob", "dtype": "bf16", "rows": 4096, "V": 131072,
         "pad": 0, "entropy": True},
        # the backward pass of a training step on a large vocabulary
        {"name": "grad_batch", "op": "grad", "dtype": "bf16", "rows": 4096, "V": 131072,
         "pad": 0, "entropy": False},
        # the same in fp32 with an odd vocabulary, an entropy bonus, and rows
        # padded to a multiple of 64
        {"name": "grad_odd_f32", "op": "grad", "dtype": "f32", "rows": 1531, "V": 50001,
         "pad": 47, "entropy": True},
        # a short prompt distilled from a few kept logits
        {"name": "distill_short_f16", "op": "distill", "dtype": "f16", "rows": 48, "V": 32768,
         "pad": 0, "K": 8, "tail": False, "masked": 5, "grad": True},
        # evaluation: the divergence alone, odd vocabulary, unaligned rows
        {"name": "distill_eval_odd_f32", "op": "distill", "dtype": "f32", "rows": 1021,
         "V": 100003, "pad": 0, "K": 50, "tail": True, "masked": 100, "grad": False},
        # training step of a student on a packed batch
        {"name": "distill_train", "op": "distill", "dtype": "bf16", "rows": 4096, "V": 131072,
         "pad": 0, "K": 64, "tail": True, "masked": 512, "grad": True},
        # policy step on one short answer
        {"name": "policy_short", "op": "policy", "dtype": "bf16", "rows": 96, "V": 32768,
         "pad": 0, "masked": 0, "ref": True, "entropy": False},
        # policy step with an entropy bonus in fp32, unaligned rows
        {"name": "policy_entropy_f32", "op": "policy", "dtype": "f32", "rows": 1024, "V": 65537,
         "pad": 0, "masked": 200, "ref": False, "entropy": True},
        # policy step on a packed batch with prompt tokens masked out
        {"name": "policy_train", "op": "policy", "dtype": "bf16", "rows": 8192, "V": 131072,
         "pad": 0, "masked": 2048, "ref": True, "entropy": False},
        # two short pairs
        {"name": "preference_short", "op": "preference", "dtype": "bf16", "rows": 150, "V": 32768,
         "pad": 0, "pairs": 2, "kind": "sigmoid", "average": False},
        # a training step on ragged pairs
        {"name": "preference_train", "op": "preference", "dtype": "bf16", "rows": 6144, "V": 65536,
         "pad": 0, "pairs": 8, "kind": "sigmoid", "average": False},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprob", "grad", "distill", "policy", "preference"])
    V = _log_uniform(rng, 1000, 262144)
    rows = _log_uniform(rng, 2 if op == "preference" else 1, min(16384, _LARGEST // V))
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if dtype == "f32" and rows * V > _LARGEST // 2:
        rows = _LARGEST // 2 // V
    case = {"op": op, "dtype": dtype, "rows": rows, "V": V, "pad": rng.choice([0, 0, -V % 64])}
    masked = rng.randrange(rows // 2 + 1)
    if op in ("logprob", "grad"):
        case["entropy"] = rng.random() < 0.5
    elif op == "distill":
        case.update(K=_log_uniform(rng, 1, 256), tail=rng.random() < 0.5, masked=masked,
                    grad=rng.random() < 0.75)
    elif op == "policy":
        case.update(masked=masked, ref=rng.random() < 0.5, entropy=rng.random() < 0.5)
    else:
        case.update(pairs=_log_uniform(rng, 1, max(1, min(64, rows // 2))),
                    kind=rng.choice(["sigmoid", "hinge", "squared"]),
                    average=rng.random() < 0.5)
    return case


def work(case):
    rows, V = case["rows"], case["V"]
    size = 4 if case["dtype"] == "f32" else 2
    live = rows - case.get("masked", 0)  # masked rows of logits need not be read
    matrix, op = V * size, case["op"]
    if op == "logprob":
        moved = rows * (matrix + 8 + 8 + 4 * case["entropy"])
    elif op == "grad":
        moved = rows * (2 * matrix + 8 + 8 + 8 * case["entropy"])
    elif op == "distill":
        moved = live * (matrix + 12 * case["K"] + 4 * case["tail"]) + rows * (8 + matrix * case["grad"])
    elif op == "policy":
        moved = live * (matrix + 16 + 4 * case["ref"]) + rows * (matrix + 8 + 4 * case["entropy"])
    else:
        moved = rows * (2 * matrix + 8) + case["pairs"] * 24
    # per element: maximum, subtract, exp, add; as many again for a gradient
    twice = op in ("grad", "preference", "policy") or case.get("grad", False)
    return {"bytes": moved, "flops": live * V * (8 if twice else 4)}


def _logits(case, g, targets):
    """Logits of a trained model: a spread of a few units and a target that
    is often among the likely tokens."""
    rows, V, pad = case["rows"], case["V"], case["pad"]
    z = torch.empty(rows, V + pad, device="cuda").normal_(0.0, 2.0, generator=g)
    lift = torch.empty(rows, 1, device="cuda").uniform_(0.0, 12.0, generator=g)
    z.scatter_add_(1, targets.unsqueeze(1), lift)
    return z.to(_TYPES[case["dtype"]])[:, :V]


def _score(z, targets):
    """Rough log-probabilities, from which the recorded ones are drawn."""
    z = z.float()
    return z.gather(1, targets.unsqueeze(1)).squeeze(1) - z.logsumexp(1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, V, op = case["rows"], case["V"], case["op"]

    def normal(*shape, std=1.0):
        return torch.empty(*shape, device="cuda").normal_(0.0, std, generator=g)

    targets = torch.randint(V, (rows,), device="cuda", generator=g)
    z = _logits(case, g, targets)
    s = {"case": case, "logits": z, "targets": targets}
    if op in ("logprob", "grad"):
        s["scale"] = 1.0 / 0.9
        s["logp"] = torch.empty(rows, device="cuda")
        s["lse"] = torch.empty(rows, device="cuda")
        s["entropy"] = torch.empty(rows, device="cuda") if case["entropy"] else None
    if op == "grad":
        x = z.double() if rows * V <= 1 << 26 else z.float()
        x = x * s["scale"]
        lse = x.logsumexp(1)
        s["lse"] = lse.float()
        if case["entropy"]:
            s["entropy"] = (lse - ((x - lse.unsqueeze(1)).exp_() * x).sum(1)).float()
        s["glogp"] = normal(rows)
        s["gentropy"] = normal(rows, std=0.01) if case["entropy"] else None
    if "masked" in case:
        keep = torch.ones(rows, device="cuda")
        keep[torch.randperm(rows, device="cuda", generator=g)[:case["masked"]]] = 0
        s["weight"] = keep / keep.sum()
    if op == "distill":
        s["scale"] = 0.5
        # the teacher agrees with the student in part
        t = z.float() + normal(rows, V, std=1.5)
        s["val"], s["idx"] = t.topk(min(case["K"], V), dim=1)
        s["teacher_lse"] = (t * s["scale"]).logsumexp(1) if case["tail"] else None
        s["row_loss"] = torch.empty(rows, device="cuda")
    if op == "policy":
        logp = _score(z, targets)
        drift = normal(rows, std=0.15)
        # the loss has a kink where a ratio meets its bound: no row sits on it
        for bound in (math.log(0.8), math.log(1.28)):
            drift = torch.where((drift - bound).abs() < 1e-3, bound + 1e-3, drift)
        s["old_logp"] = logp - drift
        s["ref_logp"] = logp + normal(rows, std=0.4) if case["ref"] else None
        s["advantage"] = normal(rows)
        s["logp"] = torch.empty(rows, device="cuda")
        s["entropy"] = torch.empty(rows, device="cuda") if case["entropy"] else None
        s["coef"] = {"clip_low": 0.2, "clip_high": 0.28, "kl_coef": 0.04 if case["ref"] else 0.0,
                     "entropy_coef": 0.01 if case["entropy"] else 0.0}
    if op == "preference":
        n = 2 * case["pairs"]
        cuts = torch.randperm(rows - 1, device="cuda", generator=g)[:n - 1].sort().values + 1
        s["starts"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows)])
        ref = _segment_sums(_score(z, targets).double(), s["starts"])
        s["ref_logp"] = (ref + normal(n, std=3.0)).float()
        if case["average"]:
            s["ref_logp"] /= (s["starts"][1:] - s["starts"][:-1])
        s["seq_logp"] = torch.empty(n, device="cuda")
    s["loss"] = torch.zeros(1, device="cuda")
    if op in ("grad", "policy", "preference") or case.get("grad"):
        s["dlogits"] = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device="cuda")
    return s


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


# --- the library's entry points -------------------------------------------------

def _own(s):
    import fp32_reductions_amd as red

    case = s["case"]
    op, dtype = case["op"], case["dtype"]
    if op == "logprob":
        getattr(red, "token_logprob_" + dtype)(
            s["logits"], s["targets"], s["logp"], s["lse"], entropy=s["entropy"], scale=s["scale"])
        return {"logp": s["logp"], "lse": s["lse"], "entropy": s["entropy"]}
    if op == "grad":
        getattr(red, "token_logprob_grad_" + dtype)(
            s["logits"], s["targets"], s["lse"], s["glogp"], s["dlogits"], entropy=s["entropy"],
            gentropy=s["gentropy"], scale=s["scale"])
        return {"dlogits": s["dlogits"]}
    if op == "distill":
        getattr(red, "distill_topk_" + dtype)(
            s["logits"], s["idx"], s["val"], s["loss"], dlogits=s.get("dlogits"),
            teacher_lse=s["teacher_lse"], weight=s["weight"], row_loss=s["row_loss"],
            scale=s["scale"])
        return {"loss": s["loss"], "row_loss": s["row_loss"], "dlogits": s.get("dlogits")}
    if op == "policy":
        getattr(red, "policy_loss_" + dtype)(
            s["logits"], s["targets"], s["old_logp"], s["advantage"], s["loss"], s["logp"],
            dlogits=s["dlogits"], ref_logp=s["ref_logp"], weight=s["weight"],
            entropy=s["entropy"], **s["coef"])
        return {"loss": s["loss"], "logp": s["logp"], "entropy": s["entropy"],
                "dlogits": s["dlogits"]}
    getattr(red, "preference_loss_" + dtype)(
        s["logits"], s["targets"], s["starts"], s["loss"], s["seq_logp"], dlogits=s["dlogits"],
        ref_logp=s["ref_logp"], kind=case["kind"], beta=0.1, average=case["average"])
    return {"loss": s["loss"], "seq_logp": s["seq_logp"], "dlogits": s["dlogits"]}


# --- the plain forms ------------------------------------------------------------

def _softmax(z, scale):
    """(scaled logits minus the row's maximum, their exponentials, the sum of
    those, the maximum)."""
    x = z.float() * scale
    m = x.amax(1, keepdim=True)
    x = x - m
    e = x.exp()
    return x, e, e.sum(1, keepdim=True), m


def _at(x, targets):
    return x.gather(1, targets.unsqueeze(1))


def _minus_onehot(p, targets):
    """p - 1 in the target's column (p is overwritten)."""
    return p.scatter_add_(1, targets.unsqueeze(1), p.new_full((p.shape[0], 1), -1.0))


def _segment_sums(v, starts):
    """fp64 sums of v over [starts[i], starts[i + 1])."""
    run_ = torch.cat([v.new_zeros(1), v.cumsum(0)])
    return run_[starts[1:]] - run_[starts[:-1]]


def _plain_logprob(s):
    x, e, total, m = _softmax(s["logits"], s["scale"])
    ln = total.log()
    out = {"logp": (_at(x, s["targets"]) - ln).squeeze(1), "lse": (m + ln).squeeze(1),
           "entropy": None}
    if s["case"]["entropy"]:
        out["entropy"] = (ln - (e * x).sum(1, keepdim=True) / total).squeeze(1)
    return out


def _plain_grad(s):
    logp = s["logits"].float() * s["scale"] - s["lse"].unsqueeze(1)
    p = logp.exp()
    factor = s["glogp"].unsqueeze(1)
    extra = None
    if s["case"]["entropy"]:
        extra = p * (logp + s["entropy"].unsqueeze(1)) * s["gentropy"].unsqueeze(1)
    d = _minus_onehot(p, s["targets"]) * -factor
    if extra is not None:
        d -= extra
    return {"dlogits": (d * s["scale"]).to(s["logits"].dtype)}


def _plain_distill(s):
    z, idx, scale, weight = s["logits"], s["idx"], s["scale"], s["weight"].unsqueeze(1)
    x, e, total, _ = _softmax(z, scale)
    t = s["val"] * scale
    if s["case"]["tail"]:
        logq = t - s["teacher_lse"].unsqueeze(1)
    else:
        logq = t - t.amax(1, keepdim=True)
        logq = logq - logq.exp().sum(1, keepdim=True).log()
    q = logq.exp()
    row = (q * (logq - x.gather(1, idx) + total.log())).sum(1, keepdim=True)
    p = e / total
    if s["case"]["tail"]:
        rest = (1.0 - q.double().sum(1, keepdim=True)).float().clamp_min(0.0)
        at = p.gather(1, idx)
        outside = p.clone().scatter_(1, idx, 0.0)
        left = outside.sum(1, keepdim=True)
        row = row + torch.where(rest > 0, rest * (rest.log() - left.log()), 0.0)
        d = (outside * (1.0 - rest / left)).scatter_(1, idx, at - q)
    else:
        d = p.scatter_add_(1, idx, -q)
    row = torch.where(weight != 0, row, 0.0)
    loss = (row.double() * weight.double()).sum().float().reshape(1)
    out = {"loss": loss, "row_loss": row.squeeze(1), "dlogits": None}
    if s["case"]["grad"]:
        out["dlogits"] = (d * (weight * scale)).to(z.dtype)
    return out


def _plain_policy(s):
    z, weight, c = s["logits"], s["weight"].unsqueeze(1), s["coef"]
    x, e, total, _ = _softmax(z, 1.0)
    ln = total.log()
    logp = _at(x, s["targets"]) - ln
    ratio = (logp - s["old_logp"].unsqueeze(1)).exp()
    adv = s["advantage"].unsqueeze(1)
    free = ratio * adv
    clipped = ratio.clamp(1.0 - c["clip_low"], 1.0 + c["clip_high"]) * adv
    row = -torch.minimum(free, clipped)
    g = torch.where(free <= clipped, -free, 0.0)
    if s["case"]["ref"]:
        d = s["ref_logp"].unsqueeze(1) - logp
        row = row + c["kl_coef"] * (d.exp() - d - 1.0)
        g = g + c["kl_coef"] * (1.0 - d.exp())
    p = e / total
    entropy = extra = None
    if s["case"]["entropy"]:
        entropy = ln - (p * x).sum(1, keepdim=True)
        row = row - c["entropy_coef"] * entropy
        extra = p * (x - ln + entropy) * c["entropy_coef"]
    dz = _minus_onehot(p, s["targets"]) * -g
    if extra is not None:
        dz += extra
    live = weight != 0
    loss = torch.where(live, row.double() * weight.double(), 0.0).sum().float().reshape(1)
    return {"loss": loss, "logp": torch.where(live, logp, 0.0).squeeze(1),
            "entropy": None if entropy is None else torch.where(live, entropy, 0.0).squeeze(1),
            "dlogits": (dz * weight).to(z.dtype)}


def _plain_preference(s):
    z, targets, starts, n = s["logits"], s["targets"], s["starts"], s["case"]["pairs"]
    x, e, total, _ = _softmax(z, 1.0)
    logp = (_at(x, targets) - total.log()).squeeze(1)
    seq = _segment_sums(logp.double(), starts)
    length = starts[1:] - starts[:-1]
    if s["case"]["average"]:
        seq = seq / length
    delta = seq - s["ref_logp"].double()
    delta = delta[:n] - delta[n:]
    beta, kind = 0.1, s["case"]["kind"]
    h = beta * delta
    if kind == "sigmoid":
        pair = (1.0 + (-h.abs()).exp()).log() + (-h).clamp_min(0.0)
        slope = -beta / (1.0 + h.exp())
    elif kind == "hinge":
        pair = (1.0 - h).clamp_min(0.0)
        slope = torch.where(h < 1.0, -beta, 0.0)
    else:
        pair = (delta - 0.5 / beta).square()
        slope = 2.0 * (delta - 0.5 / beta)
    loss = (pair.sum() / n).float().reshape(1)
    g = torch.cat([slope, -slope]) / n
    if s["case"]["average"]:
        g = g / length
    rows = torch.arange(z.shape[0], device=z.device)
    g = g[torch.searchsorted(starts[1:].contiguous(), rows, right=True)].float()
    d = _minus_onehot(e / total, targets) * -g.unsqueeze(1)
    return {"loss": loss, "seq_logp": seq.float(), "dlogits": d.to(z.dtype)}


_PLAIN = {"logprob": _plain_logprob, "grad": _plain_grad, "distill": _plain_distill,
          "policy": _plain_policy, "preference": _plain_preference}


# --- the definitions in 64 bits -------------------------------------------------
#
# Losses are written down in fp64 and their gradients taken by automatic
# differentiation, a block of rows at a time.

def exact(case, seed):
    s = prepare(case, seed)
    rows, V, op = case["rows"], case["V"], case["op"]
    step = max(1, (1 << 27) // V)
    blocks = [slice(a, min(rows, a + step)) for a in range(0, rows, step)]
    found = {"logp": [], "lse": [], "entropy": [], "row_loss": [], "dlogits": []}
    loss = 0.0
    pair_grad = None
    if op == "preference":
        logp = torch.cat([torch.log_softmax(s["logits"][b].double(), 1)
                          .gather(1, s["targets"][b].unsqueeze(1)).squeeze(1) for b in blocks])
        logp.requires_grad_()
        spans = [slice(a, b) for a, b in zip(s["starts"][:-1].tolist(), s["starts"][1:].tolist())]
        seq = torch.stack([logp[v].mean() if case["average"] else logp[v].sum() for v in spans])
        n = case["pairs"]
        ratio = seq - s["ref_logp"].double()
        delta = ratio[:n] - ratio[n:]
        if case["kind"] == "sigmoid":
            pair = -torch.nn.functional.logsigmoid(0.1 * delta)
        elif case["kind"] == "hinge":
            pair = torch.relu(1.0 - 0.1 * delta)
        else:
            pair = (delta - 5.0) ** 2
        loss = pair.mean()
        pair_grad, = torch.autograd.grad(loss, logp)
    for b in blocks:
        z = s["logits"][b].double().requires_grad_()
        y = s["targets"][b].unsqueeze(1)
        if op in ("logprob", "grad"):
            lp = torch.log_softmax(z * s["scale"], 1)
            at = lp.gather(1, y).squeeze(1)
            entropy = -(lp.exp() * lp).sum(1) if case["entropy"] else None
            if op == "grad":
                # the definition takes the log-sum-exp and the entropy as given
                with torch.no_grad():
                    lp = z * s["scale"] - s["lse"][b].double().unsqueeze(1)
                    p = lp.exp()
                    d = -p * s["glogp"][b].double().unsqueeze(1)
                    if case["entropy"]:
                        d -= (s["gentropy"][b].double().unsqueeze(1) * p
                              * (lp + s["entropy"][b].double().unsqueeze(1)))
                    d.scatter_add_(1, y, s["glogp"][b].double().unsqueeze(1))
                    found["dlogits"].append(d * s["scale"])
                continue
            found["logp"].append(at.detach())
            found["lse"].append((s["logits"][b].double() * s["scale"]).logsumexp(1))
            if case["entropy"]:
                found["entropy"].append(entropy.detach())
            continue
        lp = torch.log_softmax(z * s.get("scale", 1.0), 1)
        if op == "preference":
            at = lp.gather(1, y).squeeze(1)
            d, = torch.autograd.grad((at * pair_grad[b]).sum(), z)
            found["dlogits"].append(d)
            continue
        w = s["weight"][b].double()
        live = w != 0
        if op == "distill":
            idx, t = s["idx"][b], s["val"][b].double() * s["scale"]
            if case["tail"]:
                lq = t - s["teacher_lse"][b].double().unsqueeze(1)
            else:
                lq = torch.log_softmax(t, 1)
            q = lq.exp()
            row = (q * (lq - lp.gather(1, idx))).sum(1)
            if case["tail"]:
                rest = (1.0 - q.sum(1)).clamp_min(0.0)
                left = lp.scatter(1, idx, -math.inf).logsumexp(1)
                row = row + torch.special.xlogy(rest, rest) - torch.where(rest > 0, rest * left, 0.0)
            row = torch.where(live, row, 0.0)
            found["row_loss"].append(row.detach())
        else:
            c = s["coef"]
            at = lp.gather(1, y).squeeze(1)
            ratio, adv = (at - s["old_logp"][b].double()).exp(), s["advantage"][b].double()
            row = -torch.minimum(ratio * adv,
                                 ratio.clamp(1 - c["clip_low"], 1 + c["clip_high"]) * adv)
            if case["ref"]:
                k = s["ref_logp"][b].double() - at
                row = row + c["kl_coef"] * (torch.expm1(k) - k)
            if case["entropy"]:
                entropy = -(lp.exp() * lp).sum(1)
                row = row - c["entropy_coef"] * entropy
                found["entropy"].append(torch.where(live, entropy, 0.0).detach())
            found["logp"].append(torch.where(live, at, 0.0).detach())
        total = (torch.where(live, row, 0.0) * w).sum()
        loss = loss + total.detach()
        if "dlogits" in s:
            d, = torch.autograd.grad(total, z)
            found["dlogits"].append(d)
    found = {k: torch.cat(v) if v else None for k, v in found.items()}
    if op == "logprob":
        return {k: found[k] for k in ("logp", "lse", "entropy")}
    if op == "grad":
        return {"dlogits": found["dlogits"]}
    found["loss"] = loss.detach().reshape(1)
    if op == "distill":
        return {k: found[k] for k in ("loss", "row_loss", "dlogits")}
    if op == "policy":
        return {k: found[k] for k in ("loss", "logp", "entropy", "dlogits")}
    return {"loss": found["loss"], "seq_logp": seq.detach(), "dlogits": found["dlogits"]}
