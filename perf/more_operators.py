"""The cases on which a mixture-of-experts model's training step is measured
beyond its products: the router with scores, a bias for balance and groups of
experts, its gradient and the bias's update; and the update of the weights'
matrices by an orthogonalised momentum, with the step that applies it.  Each
case runs either in its plain form (elementary torch operations) or, with
``own``, through the binding's entry points.

Sizes: hidden 4096 and ffn 14336 are the ones of this repository's own layer;
the others are generic.
"""
import math

import torch

own = False

COEFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
MU = 0.95
EPS = 1e-7
RATE = 1e-3


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token at a server, many experts in groups
        dict(name="route_one_token", op="route", tokens=1, experts=256, top=8, score="sigmoid",
             bias=True, groups=8, kept=4, group_top=2, renorm=True, scale=2.5, fp32=True,
             train=False),
        # a decode step's tokens, few experts of an odd number, no groups
        dict(name="route_decode", op="route", tokens=48, experts=60, top=4, score="softmax",
             bias=True, groups=1, kept=1, group_top=1, renorm=False, scale=1.0, fp32=False,
             train=False),
        # a training batch: choice, gradient of the logits, update of the bias
        dict(name="route_train", op="route", tokens=16384, experts=256, top=8, score="sigmoid",
             bias=True, groups=8, kept=4, group_top=2, renorm=True, scale=2.5, fp32=True,
             train=True),
        # the same with softmax scores in bf16 whose group counts by its best expert
        dict(name="route_train_softmax", op="route", tokens=8191, experts=160, top=6,
             score="softmax", bias=False, groups=8, kept=3, group_top=1, renorm=False, scale=16.0,
             fp32=False, train=True),
        # a large batch over very many experts without groups
        dict(name="route_train_large", op="route", tokens=40000, experts=384, top=8,
             score="sigmoid", bias=True, groups=1, kept=1, group_top=2, renorm=True, scale=2.0,
             fp32=True, train=True),
        # a router's own weights: few rows, long
        dict(name="muon_router", op="muon", batch=1, rows=64, cols=4096, fp32=True),
        # one small square projection
        dict(name="muon_square", op="muon", batch=1, rows=1024, cols=1024, fp32=True),
        # a few odd matrices, gradients in bf16
        dict(name="muon_odd", op="muon", batch=3, rows=777, cols=1290, fp32=False),
        # the stacked projections of many small experts
        dict(name="muon_experts", op="muon", batch=64, rows=1024, cols=2048, fp32=True),
        # the up projection of this repository's layer
        dict(name="muon_layer", op="muon", batch=1, rows=14336, cols=4096, fp32=True),
        # a router's weights take their update, with the amax of the result
        dict(name="apply_router", op="apply", count=64 * 4096),
        # the same for the up projection
        dict(name="apply_layer", op="apply", count=14336 * 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _products(batch, rows, cols):
    """Multiply-adds of the steps' products, each done whole."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * batch * (2 * m * m * n + m ** 3)


def draw(rng):
    op = rng.choice(("route", "route", "muon", "muon", "muon", "apply"))
    if op == "apply":
        return dict(op=op, count=4 * _log(rng, 256, 14336 * 1024))
    if op == "muon":
        while True:
            batch, rows, cols = _log(rng, 1, 64), _log(rng, 16, 14336), _log(rng, 16, 14336)
            if (_products(batch, rows, cols) <= _products(1, 14336, 4096)
                    and batch * rows * cols <= 64 * 1024 * 2048):
                return dict(op=op, batch=batch, rows=rows, cols=cols, fp32=rng.random() < 0.5)
    while True:
        groups = rng.choice((1, 1, 2, 4, 8, 16))
        size = _log(rng, 2, 512)
        if groups * size <= 512:
            break
    experts = groups * size
    kept = rng.randint(1, groups)
    top = rng.randint(1, min(16, kept * size))
    return dict(op=op, tokens=min(_log(rng, 1, 65536), 40000 * 384 // experts), experts=experts,
                top=top, score=rng.choice(("sigmoid", "softmax")), bias=rng.random() < 0.7,
                groups=groups, kept=kept, group_top=rng.randint(1, 2),
                renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5, 16.0)),
                fp32=rng.random() < 0.6, train=rng.random() < 0.6)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gradient(g, batch, rows, cols):
    """A weight's gradient: a falling spectrum over some directions, noise, and
    a few large channels."""
    r = min(rows, cols, 48)
    fall = torch.arange(1, r + 1, device="cuda") ** -0.5
    a = torch.randn(batch, rows, r, generator=g, device="cuda") * fall
    b = torch.randn(batch, r, cols, generator=g, device="cuda")
    x = torch.bmm(a, b)
    x += torch.randn(batch, rows, cols, generator=g, device="cuda")
    x *= 1 + 9 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
    return x * 0.01


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        # an uneven preference of the experts, some masked, some padding tokens
        x = torch.randn(t, e, generator=g, device="cuda") * 1.5
        x += torch.randn(e, generator=g, device="cuda") * 0.7
        masked = torch.rand(t, e, generator=g, device="cuda") < 0.05
        masked |= torch.rand(t, 1, generator=g, device="cuda") < 0.03
        x = x.masked_fill(masked, -math.inf)
        s["logits"] = x if case["fp32"] else x.bfloat16()
        s["bias"] = None
        if case["bias"]:
            spread = 0.05 if case["score"] == "sigmoid" else 0.2 / e
            s["bias"] = torch.randn(e, generator=g, device="cuda") * spread
        if case["train"]:
            s["dweight"] = torch.randn(t, case["top"], generator=g, device="cuda")
    elif case["op"] == "muon":
        shape = case["batch"], case["rows"], case["cols"]
        x = _gradient(g, *shape)
        s["momentum"] = 3 * x + 2 * _gradient(g, *shape)
        s["grad"] = x if case["fp32"] else x.bfloat16()
    else:
        n = case["count"]
        s["weight"] = torch.randn(n, generator=g, device="cuda") / 64
        s["update"] = (torch.randn(n, generator=g, device="cuda") / 64).bfloat16()
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from nvfp4_block_scaled_03_gb300 import binding as nv
    case = s["case"]
    if case["op"] == "route":
        how = dict(score=nv.SCORE_SIGMOID if case["score"] == "sigmoid" else nv.SCORE_SOFTMAX,
                   renormalise=case["renorm"], scale=case["scale"])
        p = nv.nvfp4_route_scored_fwd(s["logits"], case["top"], bias=s["bias"],
                                      groups=case["groups"], groups_kept=case["kept"],
                                      group_top=case["group_top"], **how)
        got = dict(expert=p.expert, weight=p.weight, sizes=p.sizes, offsets=p.offsets, row=p.row,
                   source=p.source)
        if case["train"]:
            got["dlogits"] = nv.nvfp4_route_scored_bwd(s["logits"], p, s["dweight"], **how)
            if s["bias"] is not None:
                got["bias"] = nv.nvfp4_route_balance(p.sizes, s["bias"], RATE)
        return got
    if case["op"] == "muon":
        update = nv.nvfp4_muon_update(s["grad"], s["momentum"], mu=MU, nesterov=True,
                                      coefs=COEFS, steps=STEPS, eps=EPS)
        return dict(update=update, momentum=s["momentum"])
    amax = nv.nvfp4_muon_apply(s["weight"], s["update"], lr=0.01, scale=0.2 * 14336 ** 0.5,
                               decay=0.1)
    return dict(weight=s["weight"], amax=amax)


def _plain_route(s):
    case = s["case"]
    top, groups = case["top"], case["groups"]
    # 64 bits: two experts' scores may lie closer than 32 bits tell apart
    x = s["logits"].double()
    t, e = x.shape
    open_ = x > -math.inf
    if case["score"] == "sigmoid":
        score = torch.where(open_, 1 / (1 + torch.exp(-x)), 0.0)
    else:
        most = x.amax(1, keepdim=True)
        ex = torch.exp(x - torch.where(most > -math.inf, most, 0.0))
        total = ex.sum(1, keepdim=True)
        score = ex / torch.where(total > 0, total, 1.0)
    key = score if s["bias"] is None else score + s["bias"].double()
    key = torch.where(open_, key, -math.inf)
    if groups > 1:
        best = torch.sort(key.view(t, groups, -1), dim=2, descending=True).values
        best = best[:, :, :case["group_top"]]
        worth = torch.where(best > -math.inf, best, 0.0).sum(2)
        worth = torch.where(best[:, :, 0] > -math.inf, worth, -math.inf)
        order = torch.argsort(worth, dim=1, descending=True, stable=True)
        keep = torch.zeros(t, groups, dtype=torch.bool, device=x.device)
        keep.scatter_(1, order[:, :case["kept"]], True)
        key = torch.where(keep.repeat_interleave(e // groups, 1), key, -math.inf)
    value, index = torch.sort(key, dim=1, descending=True, stable=True)
    some = value[:, :top] > -math.inf
    at = index[:, :top]
    expert = torch.where(some, at, -1)
    chosen = torch.where(some, score.gather(1, at), 0.0)
    total = chosen.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(chosen[:, :1])
    share = chosen / torch.where(total > 0, total, 1.0)
    weight = case["scale"] * share

    flat = torch.where(some, at, e).reshape(-1)
    order = torch.argsort(flat, stable=True)
    count = torch.zeros(e + 1, dtype=torch.int64, device=x.device)
    count.scatter_add_(0, flat, torch.ones_like(flat))
    first = torch.cumsum(count, 0) - count
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(t * top, device=x.device) - first[flat[order]]
    sizes = count[:e]
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=x.device)
    offsets[1:] = torch.cumsum((sizes + 127) // 128 * 128, 0)
    row = torch.where(flat < e, offsets[flat] + rank, -1)
    rows = _rows_bound(t * top, e)
    source = torch.full((rows + 1,), -1, dtype=torch.int64, device=x.device)
    source[torch.where(row < 0, rows, row)] = torch.arange(t * top, device=x.device)
    i = torch.int32
    got = dict(expert=expert.to(i), weight=weight.float(), sizes=sizes.to(i),
               offsets=offsets.to(i), row=row.reshape(t, top).to(i), source=source[:rows].to(i))
    if case["train"]:
        dw = torch.where(some, s["dweight"].double(), 0.0) * case["scale"]
        if case["renorm"]:
            ds = share * (dw - (share * dw).sum(1, keepdim=True))
        else:
            ds = share * dw
        dl = torch.zeros_like(x)
        if case["score"] == "sigmoid":
            dl.scatter_add_(1, at, ds * (1 - chosen))
        else:
            if not case["renorm"]:
                dl -= score * ds.sum(1, keepdim=True)
            dl.scatter_add_(1, at, ds)
        got["dlogits"] = dl.to(s["logits"].dtype)
        if s["bias"] is not None:
            gap = t * top - (flat == e).sum() - sizes * e  # of the mean over a load, times e
            got["bias"] = s["bias"].add_(RATE * torch.sign(gap).float())
    return got


def _plain_muon(s):
    a, b, c = COEFS
    grad = s["grad"].float()
    buf = s["momentum"].mul_(MU).add_(grad)
    x = grad + MU * buf
    x = x / x.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt().clamp(min=EPS).float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if tall:
        x = x.transpose(1, 2)
    return dict(update=x.bfloat16().contiguous(), momentum=buf)


def _plain_apply(s):
    w = s["weight"]
    w.mul_(1 - 0.01 * 0.1).sub_((0.01 * 0.2 * 14336 ** 0.5) * s["update"].float())
    return dict(weight=w, amax=w.abs().max().reshape(1))


_PLAIN = dict(route=_plain_route, muon=_plain_muon, apply=_plain_apply)


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------
def _exact_route(s):
    """Weights and logits' gradient: the choice as a mask over all experts, and
    the gradient by autograd."""
    case = s["case"]
    t, e = s["logits"].shape
    closed = s["logits"] == -math.inf
    x = s["logits"].double().masked_fill(closed, 0.0).requires_grad_(case["train"])
    if case["score"] == "sigmoid":
        score = torch.sigmoid(x)
    else:
        # a row without an open expert has no score
        score = torch.exp(torch.log_softmax(x.masked_fill(closed, -1e300), 1))
    score = score * ~closed
    value = score.detach() + (0.0 if s["bias"] is None else s["bias"].double())
    value = value.masked_fill(closed, -math.inf)
    if case["groups"] > 1:
        parts = value.reshape(t, case["groups"], e // case["groups"])
        k = min(case["group_top"], parts.shape[2])
        worth = parts.topk(k, 2).values
        dead = worth[:, :, 0] == -math.inf
        worth = worth.masked_fill(worth == -math.inf, 0.0).sum(2).masked_fill(dead, -math.inf)
        rank = torch.argsort(torch.argsort(-worth, dim=1, stable=True), dim=1, stable=True)
        out = (rank >= case["kept"]).unsqueeze(2).expand_as(parts)
        value = parts.masked_fill(out, -math.inf).reshape(t, e)
    at = torch.argsort(-value, dim=1, stable=True)[:, :case["top"]]
    live = torch.gather(value, 1, at) > -math.inf
    weight = torch.gather(score, 1, at) * live
    if case["renorm"]:
        weight = weight / weight.sum(1, keepdim=True).masked_fill(~live.any(1, keepdim=True), 1.0)
    weight = weight * case["scale"]
    got = dict(weight=weight.detach())
    if case["train"]:
        (weight * s["dweight"].double()).sum().backward()
        got["dlogits"] = x.grad
        if s["bias"] is not None:
            load = torch.bincount(at[live], minlength=e).double()
            got["bias"] = s["bias"].double() + RATE * torch.sign(load.mean() - load).round()
    return got


def _exact_muon(s):
    """Each matrix by itself, the polynomial on the side of the columns or rows
    that has fewer, in Horner's form."""
    a, b, c = COEFS
    shape = s["grad"].shape
    update = torch.empty(shape, dtype=torch.float64, device="cuda")
    momentum = torch.empty(shape, dtype=torch.float64, device="cuda")
    for i in range(shape[0]):
        grad = s["grad"][i].double()
        momentum[i] = MU * s["momentum"][i].double() + grad
        x = grad + MU * momentum[i]
        x = x / max(float(torch.linalg.matrix_norm(x)), EPS)
        one = torch.eye(min(x.shape), dtype=torch.float64, device="cuda")
        for _ in range(STEPS):
            if x.shape[0] > x.shape[1]:
                p = x.t() @ x
                x = x @ (a * one + p @ (b * one + c * p))
            else:
                p = x @ x.t()
                x = (a * one + p @ (b * one + c * p)) @ x
        update[i] = x
    return dict(update=update, momentum=momentum)


def _exact_apply(s):
    w = s["weight"].double() * (1 - 0.01 * 0.1)
    w = w - 0.01 * (0.2 * math.sqrt(14336)) * s["update"].double()
    return dict(weight=w, amax=torch.maximum(w.max(), -w.min()).reshape(1))


def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, muon=_exact_muon, apply=_exact_apply)[case["op"]](s)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def _rows_bound(assignments, experts):
    """Rows that hold every expert's rows padded to whole blocks of 128."""
    return (assignments + 127 * min(experts, assignments)) // 128 * 128


def work(case):
    if case["op"] == "apply":
        # the weight read and written, the update read
        return dict(bytes=10 * case["count"] + 4, flops=4 * case["count"])
    if case["op"] == "muon":
        batch, rows, cols = case["batch"], case["rows"], case["cols"]
        m, n = min(rows, cols), max(rows, cols)
        # Gram matrix and its square are symmetric: half of each
        return dict(bytes=batch * m * n * ((4 if case["fp32"] else 2) + 4 + 4 + 2),
                    flops=STEPS * batch * (m * m * n + m ** 3 + 2 * m * m * n))
    t, e, top = case["tokens"], case["experts"], case["top"]
    wide = 4 if case["fp32"] else 2
    out = t * top * 12 + 4 * (2 * e + 1) + 4 * _rows_bound(t * top, e)
    moved = t * e * wide + out + (4 * e if case["bias"] else 0)
    if case["train"]:
        moved += t * e * wide + 4 * t * top + (4 * e if case["bias"] else 0)
    return dict(bytes=moved, flops=t * e * (10 if case["train"] else 6))
