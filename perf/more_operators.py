"""Measured cases of the operators around the last layer of a model.

Four operators of a training step's end, each a reduction over rows beside the
losses over rows of logits:

    norm       the root-mean-square norm of a row and its residual's sum, in the
               row's type or in 8 bits with a scale for each row
    norm_grad  its gradient: rows, and the column sums of the weight's
    router     the balance loss of a router's logits, its counts of the rows of
               each expert, and the gradient
    head       the cross entropy of hidden rows against an output layer, whose
               logits are made and reduced in pieces of the vocabulary and never
               kept, with the gradients of the rows and of the layer

Each case is one pass of one operator.  ``own`` selects the library's entry
points; otherwise the operators are computed by elementary torch operations in
fp32 (sums over many rows in fp64), rounded once at the end.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_E4M3 = torch.float8_e4m3fn
_E4M3_MAX = 448.0
_LARGEST = 1 << 29   # logits of the largest output layer's pass
_PRODUCT = 1 << 41   # rows x vocabulary x width of the largest


def listed():
    return [
        # one token of a sequence that is being generated, quantised for an 8-bit product
        {"name": "norm_one_token", "op": "norm", "dtype": "bf16", "rows": 1, "D": 4096, "pad": 0,
         "residual": True, "bits8": True},
        # a batch of prompts before an 8-bit product
        {"name": "norm_prompts_8bit", "op": "norm", "dtype": "bf16", "rows": 8192, "D": 8192,
         "pad": 0, "residual": True, "bits8": True},
        # fp32 rows of odd width, unaligned
        {"name": "norm_odd_f32", "op": "norm", "dtype": "f32", "rows": 1531, "D": 5003, "pad": 0,
         "residual": False, "bits8": False},
        # the backward pass of a training step, with the gradient that arrives past the norm
        {"name": "norm_grad_train", "op": "norm_grad", "dtype": "bf16", "rows": 16384, "D": 4096,
         "pad": 0, "residual": True},
        # a router's losses on a short prompt
        {"name": "router_short", "op": "router", "dtype": "bf16", "rows": 96, "E": 8, "K": 2,
         "masked": 5, "z": True, "grad": True},
        # a router with many experts in a training step, padding masked
        {"name": "router_train_f32", "op": "router", "dtype": "f32", "rows": 65536, "E": 128,
         "K": 8, "masked": 4096, "z": True, "grad": True},
        # an odd number of experts, 16-bit logits
        {"name": "router_odd", "op": "router", "dtype": "bf16", "rows": 16384, "E": 61, "K": 6,
         "masked": 0, "z": False, "grad": True},
        # scoring one token while a sequence is generated
        {"name": "head_one_token", "op": "head", "dtype": "bf16", "rows": 1, "V": 32768,
         "D": 4096, "masked": 0, "z": False, "grad": False},
        # evaluation of a text with its prompt masked, odd vocabulary
        {"name": "head_eval_odd", "op": "head", "dtype": "bf16", "rows": 1021, "V": 50001,
         "D": 2048, "masked": 100, "z": False, "grad": False},
        # a step on one short text
        {"name": "head_short_train", "op": "head", "dtype": "bf16", "rows": 96, "V": 32768,
         "D": 2048, "masked": 5, "z": False, "grad": True},
        # half precision, odd vocabulary and width, the log-sum-exp held near 0
        {"name": "head_odd_train_f16", "op": "head", "dtype": "f16", "rows": 1531, "V": 65537,
         "D": 1000, "masked": 200, "z": True, "grad": True},
        # a training step on a large vocabulary, an eighth of the rows masked
        {"name": "head_train", "op": "head", "dtype": "bf16", "rows": 4096, "V": 131072,
         "D": 4096, "masked": 512, "z": False, "grad": True},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "router", "head", "head"])
    if op in ("norm", "norm_grad"):
        D = _log_uniform(rng, 128, 16384)
        D -= D % rng.choice([1, 8, 64, 128])
        rows = _log_uniform(rng, 1, min(65536, (1 << 26) // D))
        case = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16", "bf16"]), "rows": rows,
                "D": D, "pad": rng.choice([0, 0, 64]), "residual": rng.random() < 0.6}
        if op == "norm":
            case["bits8"] = rng.random() < 0.5
        return case
    dtype = rng.choice(["f16", "bf16", "bf16"])
    if op == "router":
        E = _log_uniform(rng, 4, 512)
        rows = _log_uniform(rng, 1, min(131072, (1 << 25) // E))
        return {"op": op, "dtype": rng.choice(["f32", dtype]), "rows": rows, "E": E,
                "K": rng.randint(1, min(8, E)), "masked": rng.randrange(rows // 2 + 1),
                "z": rng.random() < 0.5, "grad": rng.random() < 0.75}
    V = _log_uniform(rng, 1000, 262144)
    D = 8 * _log_uniform(rng, 16, 1024)
    rows = _log_uniform(rng, 1, min(8192, _LARGEST // V, _PRODUCT // (V * D)))
    return {"op": op, "dtype": dtype, "rows": rows, "V": V, "D": D,
            "masked": rng.randrange(rows // 2 + 1), "z": rng.random() < 0.5,
            "grad": rng.random() < 0.6}


def work(case):
    op, rows = case["op"], case["rows"]
    size = 4 if case["dtype"] == "f32" else 2
    live = rows - case.get("masked", 0)
    if op == "norm":
        D, both = case["D"], 2 if case["residual"] else 1
        out = (1 + 4 / D if case["bits8"] else size) + (size if case["residual"] else 0)
        return {"bytes": rows * (D * (both * size + out) + 4) + D * size, "flops": 6 * rows * D}
    if op == "norm_grad":
        D, read = case["D"], 3 if case["residual"] else 2
        return {"bytes": rows * (D * size * (read + 1) + 4) + D * (size + 4),
                "flops": 10 * rows * D}
    if op == "router":
        E = case["E"]
        moved = live * (E * size + 8 * case["K"]) + rows * (4 + E * size * case["grad"]) + E * 12
        return {"bytes": moved, "flops": live * E * (9 if case["grad"] else 5)}
    # the products of hidden rows and layer, and of the two gradients; a fourth,
    # of the logits again, is the price of not keeping them
    V, D = case["V"], case["D"]
    both = 2 if case["grad"] else 1
    return {"bytes": both * V * D * size + live * D * size * both + rows * 20,
            "flops": 2 * live * V * D * (3 if case["grad"] else 1)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, dtype = case["op"], case["rows"], _TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.empty(*shape, device="cuda").normal_(0.0, std, generator=g)

    def matrix(std):
        """rows x D in the case's type, rows `pad` elements apart."""
        D = case["D"]
        return normal(rows, D + case["pad"], std=std).to(dtype)[:, :D]

    def like(m):
        return torch.empty_strided(m.shape, m.stride(), dtype=m.dtype, device="cuda")

    s = {"case": case}
    if op in ("norm", "norm_grad"):
        D = case["D"]
        s["weight"] = (1.0 + normal(D, std=0.2)).to(dtype)
        s["rstd"] = torch.empty(rows, device="cuda")
    if op == "norm":
        s["eps"] = 1e-6
        # a block's output, and the residual stream, in which some columns run high
        s["x"] = matrix(1.0)
        s["residual"] = s["sum"] = None
        if case["residual"]:
            high = 1.0 + 20.0 * (torch.rand(D, device="cuda", generator=g) < 0.01).float()
            s["residual"] = like(s["x"]).copy_(matrix(2.0).float() * high)
            s["sum"] = like(s["x"])
        s["y"] = torch.empty(rows, D, dtype=_E4M3 if case["bits8"] else dtype, device="cuda")
        s["yscale"] = torch.empty(rows, device="cuda") if case["bits8"] else None
    elif op == "norm_grad":
        s["h"] = matrix(2.0)
        s["rstd"] = (s["h"].double().square().mean(1) + 1e-6).rsqrt().float()
        s["dy"] = matrix(0.01)
        s["dsum"] = matrix(0.01) if case["residual"] else None
        s["dx"] = like(s["h"])
        s["dweight"] = torch.empty(D, device="cuda")
    else:
        keep = torch.ones(rows, device="cuda")
        keep[torch.randperm(rows, device="cuda", generator=g)[:case["masked"]]] = 0
        # half precision trains with a factor on the loss that keeps small gradients in range
        s["row_weight"] = keep / keep.sum() * (1024.0 if case["dtype"] == "f16" else 1.0)
        s["loss"] = torch.zeros(1, device="cuda")
    if op == "router":
        E = case["E"]
        # a router that has come to like some of its experts
        logits = normal(rows, E, std=1.5) + normal(E, std=0.7)
        s["logits"] = logits.to(dtype)
        s["experts"] = s["logits"].float().topk(case["K"], dim=1).indices
        s["counts"] = torch.empty(E, dtype=torch.int64, device="cuda")
        s["prob"] = torch.empty(E, device="cuda")
        s["dlogits"] = like(s["logits"]) if case["grad"] else None
        s["balance"], s["z"] = 0.01, 0.001 if case["z"] else 0.0
    elif op == "head":
        V, D = case["V"], case["D"]
        s["weight"] = normal(V, D, std=2.0 / math.sqrt(D)).to(dtype)
        s["targets"] = torch.randint(V, (rows,), device="cuda", generator=g)
        # rows after the last norm; a trained model's target is often likely
        lift = torch.empty(rows, 1, device="cuda").uniform_(0.0, 12.0, generator=g)
        at = s["weight"][s["targets"]].float()
        s["hidden"] = (normal(rows, D) + at * (lift / at.square().sum(1, keepdim=True))).to(dtype)
        s["z"] = 1e-4 if case["z"] else 0.0
        s["logp"] = torch.empty(rows, device="cuda")
        s["lse"] = torch.empty(rows, device="cuda")
        s["dhidden"] = like(s["hidden"]) if case["grad"] else None
        s["dweight"] = like(s["weight"]) if case["grad"] else None
    return s


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


# --- the library's entry points -------------------------------------------------

def _own(s):
    import fp32_reductions_amd as red

    op, dtype = s["case"]["op"], s["case"]["dtype"]
    if op == "norm":
        getattr(red, "add_rmsnorm_" + dtype)(
            s["x"], s["weight"], s["y"], residual=s["residual"], sum=s["sum"],
            yscale=s["yscale"], rstd=s["rstd"], eps=s["eps"])
        return {"y": s["y"], "yscale": s["yscale"], "sum": s["sum"], "rstd": s["rstd"]}
    if op == "norm_grad":
        getattr(red, "rmsnorm_grad_" + dtype)(
            s["h"], s["weight"], s["rstd"], s["dy"], s["dx"], dsum=s["dsum"],
            dweight=s["dweight"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "router":
        getattr(red, "router_balance_" + dtype)(
            s["logits"], s["experts"], s["loss"], s["counts"], dlogits=s["dlogits"],
            weight=s["row_weight"], prob=s["prob"], balance_coef=s["balance"], z_coef=s["z"])
        return {"loss": s["loss"], "counts": s["counts"], "prob": s["prob"],
                "dlogits": s["dlogits"]}
    getattr(red, "linear_ce_" + dtype)(
        s["hidden"], s["weight"], s["targets"], s["loss"], logp=s["logp"], lse=s["lse"],
        dhidden=s["dhidden"], dweight=s["dweight"], row_weight=s["row_weight"], z_coef=s["z"])
    return {"loss": s["loss"], "logp": s["logp"], "lse": s["lse"], "dhidden": s["dhidden"],
            "dweight": s["dweight"]}


# --- the plain forms ------------------------------------------------------------

def _plain_norm(s):
    case, dtype = s["case"], s["x"].dtype
    h = s["x"].float()
    if case["residual"]:
        h = h + s["residual"].float()
    rstd = (h.square().mean(1) + s["eps"]).rsqrt()
    y = h * rstd.unsqueeze(1) * s["weight"].float()
    out = {"y": None, "yscale": None, "sum": h.to(dtype) if case["residual"] else None,
           "rstd": rstd}
    if not case["bits8"]:
        out["y"] = y.to(dtype)
        return out
    most = y.abs().amax(1)
    out["yscale"] = most / _E4M3_MAX
    inverse = torch.where(most > 0, _E4M3_MAX / most, 0.0)
    out["y"] = (y * inverse.unsqueeze(1)).to(_E4M3)
    return out


def _plain_norm_grad(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
    n = h * rstd
    g = dy * s["weight"].float()
    dx = (g - n * (g * n).mean(1, keepdim=True)) * rstd
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * n).double().sum(0).float()}


def _plain_router(s):
    case, w = s["case"], s["row_weight"].unsqueeze(1)
    E = case["E"]
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(1, keepdim=True)
    lse, p = m + total.log(), e / total
    live = s["row_weight"] != 0
    counts = torch.zeros(E, dtype=torch.int64, device=x.device)
    chosen = live.to(torch.int64).unsqueeze(1).expand(-1, case["K"])
    counts.scatter_add_(0, s["experts"].reshape(-1), chosen.reshape(-1))
    share = counts.double() / counts.sum().clamp_min(1)
    prob = (p * w).double().sum(0)
    loss = s["balance"] * E * (share * prob).sum()
    loss = loss + s["z"] * (w.double() * lse.double().square()).sum()
    out = {"loss": loss.float().reshape(1), "counts": counts, "prob": prob.float(),
           "dlogits": None}
    if case["grad"]:
        c = (s["balance"] * E * share).float()
        d = p * (c - (p * c).sum(1, keepdim=True) + 2.0 * s["z"] * lse)
        out["dlogits"] = (d * w).to(s["logits"].dtype)
    return out


def _plain_head(s):
    w, targets = s["row_weight"].unsqueeze(1), s["targets"].unsqueeze(1)
    hidden, layer = s["hidden"].float(), s["weight"].float()
    x = hidden @ layer.t()
    m = x.amax(1, keepdim=True)
    at = x.gather(1, targets)
    x = x.sub_(m).exp_()
    total = x.sum(1, keepdim=True)
    lse = m + total.log()
    logp = (at - m) - total.log()
    live = w != 0
    row = torch.where(live, lse.double().square() * s["z"] - logp.double(), 0.0)
    out = {"loss": (row * w.double()).sum().float().reshape(1),
           "logp": torch.where(live, logp, 0.0).squeeze(1),
           "lse": torch.where(live, lse, 0.0).squeeze(1), "dhidden": None, "dweight": None}
    if s["case"]["grad"]:
        x.mul_(w * (1.0 + 2.0 * s["z"] * lse) / total)
        x.scatter_add_(1, targets, -w)
        out["dhidden"] = (x @ layer).to(s["hidden"].dtype)
        out["dweight"] = (x.t() @ hidden).to(s["weight"].dtype)
    return out


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "router": _plain_router,
          "head": _plain_head}


# --- the definitions in 64 bits -------------------------------------------------
#
# Losses and norms are written down in fp64 and their gradients taken by
# automatic differentiation.  The values held in 8 bits are given before their
# rounding.

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + (s["residual"].double() if case["residual"] else 0.0)
        ms = (h * h).sum(1) / case["D"] + s["eps"]
        y = h / ms.sqrt().unsqueeze(1) * s["weight"].double()
        out = {"y": y, "yscale": None, "sum": h if case["residual"] else None,
               "rstd": 1.0 / ms.sqrt()}
        if case["bits8"]:
            out["yscale"] = y.abs().max(1).values / _E4M3_MAX
            out["y"] = y / out["yscale"].unsqueeze(1)
        return out
    if op == "norm_grad":
        # rstd is a given number here, of which the formula takes the derivative:
        # d rstd / d h = -rstd^3 h / D
        h, w = s["h"].double().requires_grad_(), s["weight"].double().requires_grad_()
        r = s["rstd"].double().unsqueeze(1)
        moved = r - r ** 3 * ((h - h.detach()) * h.detach()).sum(1, keepdim=True) / case["D"]
        y = h * moved * w
        dx, dw = torch.autograd.grad((y * s["dy"].double()).sum(), [h, w])
        return {"dx": dx if s["dsum"] is None else dx + s["dsum"].double(), "dweight": dw}
    w = s["row_weight"].double()
    live = w != 0
    if op == "router":
        z = s["logits"].double().requires_grad_()
        counts = torch.bincount(s["experts"][live].reshape(-1), minlength=case["E"])
        prob = (torch.softmax(z, 1) * w.unsqueeze(1)).sum(0)
        share = counts.double() / max(1, int(counts.sum()))
        loss = s["balance"] * case["E"] * torch.dot(share, prob)
        if case["z"]:
            loss = loss + s["z"] * torch.dot(w, torch.logsumexp(z, 1) ** 2)
        dz = torch.autograd.grad(loss, z)[0] if case["grad"] else None
        return {"loss": loss.detach().reshape(1), "counts": counts, "prob": prob.detach(),
                "dlogits": dz}
    layer = s["weight"].double()
    step = max(1, (1 << 27) // case["V"])
    found = {"logp": [], "lse": [], "dhidden": []}
    loss, dweight = 0.0, torch.zeros_like(layer) if case["grad"] else None
    for a in range(0, case["rows"], step):
        b = slice(a, a + step)
        hidden = s["hidden"][b].double()
        z = (hidden @ layer.t()).requires_grad_(case["grad"])
        lse = torch.logsumexp(z, 1)
        at = z.gather(1, s["targets"][b].unsqueeze(1)).squeeze(1)
        row = torch.where(live[b], lse - at + s["z"] * lse ** 2, 0.0)
        part = (row * w[b]).sum()
        loss = loss + part.detach()
        found["logp"].append(torch.where(live[b], at - lse, 0.0).detach())
        found["lse"].append(torch.where(live[b], lse, 0.0).detach())
        if case["grad"]:
            d, = torch.autograd.grad(part, z)
            found["dhidden"].append(d @ layer)
            dweight += d.t() @ hidden
    return {"loss": loss.reshape(1), "logp": torch.cat(found["logp"]),
            "lse": torch.cat(found["lse"]),
            "dhidden": torch.cat(found["dhidden"]) if case["grad"] else None,
            "dweight": dweight}
