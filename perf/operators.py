"""The cases on which the mixture-of-experts operators are measured: grouped
NVFP4 products with ragged groups, the norms around a block with its gate and
residual scales, the router with its plan, and the rows' way to the experts
and back.  Each case runs either in its plain form (elementary torch
operations in 32 bits) or, with ``own``, through the binding's entry points.

Sizes: hidden 4096 and ffn 14336 are the ones of this repository's own layer;
the others are generic.
"""
import math

import torch

own = False

EPS = 1e-5


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token at a server: two of eight experts' up projections, all weight traffic
        dict(name="fprop_one_token", op="fprop", experts=8, tokens=1, top=2, k=4096, n=14336),
        # a training batch's up projection, eight large experts
        dict(name="fprop_train", op="fprop", experts=8, tokens=8192, top=2, k=4096, n=14336),
        # many small experts with few rows each: ragged, most blocks partly filled
        dict(name="fprop_many_experts", op="fprop", experts=64, tokens=777, top=8, k=2048, n=1024),
        # the gradient of the up projection's input, through the transposed weights
        dict(name="dgrad_train", op="dgrad", experts=8, tokens=4096, top=2, k=14336, n=4096),
        # weight gradients folded into FP32 masters, contraction over ragged rows
        dict(name="wgrad_fold", op="wgrad", experts=8, tokens=8192, top=2, m=4096, n=2048,
             fold=True),
        # weight gradients of many small experts in bf16
        dict(name="wgrad_many_experts", op="wgrad", experts=64, tokens=4000, top=8, m=1024, n=2048,
             fold=False),
        # closing one block and opening the next for the tokens of a decode step
        dict(name="norm_decode", op="norm", tokens=16, d=4096, gate="channel", fp32=False,
             back=False),
        # the same over a training batch
        dict(name="norm_train", op="norm", tokens=16384, d=4096, gate="channel", fp32=False,
             back=False),
        # its backward, with the residual stream in FP32 and a gate per token
        dict(name="norm_train_backward", op="norm", tokens=8191, d=4096, gate="row", fp32=True,
             back=True),
        # routing the tokens of a decode step, forward only
        dict(name="route_decode", op="route", tokens=8, experts=64, top=8, chosen=True, fp32=True,
             back=False),
        # routing a training batch, with the gradient of the logits
        dict(name="route_train", op="route", tokens=16384, experts=128, top=8, chosen=False,
             fp32=False, back=True),
        # a training batch's rows to the experts and back, and both gradients
        dict(name="move_train", op="move", tokens=8192, experts=64, top=4, d=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _draw(rng)
    while 3072 in case.values():  # not a size of this repository
        case = _draw(rng)
    return case


def _draw(rng):
    op = rng.choice(("fprop", "dgrad", "wgrad", "norm", "route", "move"))
    if op in ("fprop", "dgrad", "wgrad"):
        while True:
            experts = _log(rng, 2, 128)
            top = rng.randint(1, min(8, experts))
            tokens = _log(rng, 1, 16384)
            a, b = 128 * _log(rng, 2, 112), 128 * _log(rng, 2, 112)
            if experts * a * b <= 8 * 4096 * 14336 and tokens * top * a * b <= 8192 * 2 * 4096 * 14336 \
                    and tokens * top <= 65536:
                break
        if op == "wgrad":
            return dict(op=op, experts=experts, tokens=tokens, top=top, m=a, n=b,
                        fold=rng.random() < 0.5)
        return dict(op=op, experts=experts, tokens=tokens, top=top, k=a, n=b)
    if op == "norm":
        d = 8 * _log(rng, 8, 2048)
        return dict(op=op, tokens=min(_log(rng, 1, 32768), 16384 * 4096 // d), d=d,
                    gate=rng.choice(("none", "channel", "row")), fp32=rng.random() < 0.5,
                    back=rng.random() < 0.5)
    experts = _log(rng, 2, 512)
    top = rng.randint(1, min(16, experts))
    if op == "route":
        return dict(op=op, tokens=_log(rng, 1, 65536), experts=experts, top=top,
                    chosen=rng.random() < 0.5, fp32=rng.random() < 0.5, back=rng.random() < 0.5)
    d = 8 * _log(rng, 8, 1024)
    return dict(op=op, tokens=max(1, min(_log(rng, 1, 16384), 8192 * 4 * 4096 // (d * top))),
                experts=experts, top=top, d=d)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _rows_bound(assignments, experts):
    """Rows that hold every expert's rows padded to whole blocks of 128."""
    return (assignments + 127 * min(experts, assignments)) // 128 * 128


def _logits(case, g):
    """Router logits as a trained router gives them: an uneven preference of
    the experts, some tokens with masked experts, and padding tokens."""
    t, e = case["tokens"], case["experts"]
    x = torch.randn(t, e, generator=g, device="cuda") * 1.5
    x += torch.randn(e, generator=g, device="cuda") * 0.7
    return x


def _plan(logits, top):
    """Expert of every slot (-1: none), and the rows' places, in torch."""
    t, e = logits.shape
    value, index = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    expert = torch.where(value[:, :top] > -math.inf, index[:, :top], -1)
    flat = torch.where(expert < 0, e, expert).reshape(-1)
    order = torch.argsort(flat, stable=True)
    count = torch.zeros(e + 1, dtype=torch.int64, device=logits.device)
    count.scatter_add_(0, flat, torch.ones_like(flat))
    first = torch.cumsum(count, 0) - count
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(t * top, device=logits.device) - first[flat[order]]
    sizes = count[:e]
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=logits.device)
    offsets[1:] = torch.cumsum((sizes + 127) // 128 * 128, 0)
    row = torch.where(flat < e, offsets[flat] + rank, -1)
    rows = _rows_bound(t * top, e)
    source = torch.full((rows + 1,), -1, dtype=torch.int64, device=logits.device)
    source[torch.where(row < 0, rows, row)] = torch.arange(t * top, device=logits.device)
    i = torch.int32
    return dict(expert=expert.to(i), sizes=sizes.to(i), offsets=offsets.to(i),
                row=row.reshape(t, top).to(i), source=source[:rows].to(i))


def _quantised(x):
    """NVFP4 codes, block scales in the layout of the tensor cores and the
    decode scale of x [rows, cols], rows and cols multiples of 128 and 64."""
    rows, cols = x.shape
    amax = x.abs().max()
    enc = torch.where(amax > 0, 2688.0 / amax.clamp(min=1e-30), torch.ones_like(amax))
    blocks = x.view(rows, cols // 16, 16)
    scale = (blocks.abs().amax(2) / 6 * enc).to(torch.float8_e4m3fn)
    s = scale.float()
    y = blocks * torch.where(s > 0, enc / s.clamp(min=1e-30), torch.zeros_like(s)).unsqueeze(2)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), edges, out_int32=True).to(torch.uint8)
    code = (code | ((y < 0).to(torch.uint8) << 3)).view(rows, cols // 2, 2)
    packed = (code[:, :, 0] | (code[:, :, 1] << 4)).contiguous()
    sw = scale.view(torch.uint8).view(rows // 128, 4, 32, cols // 64, 4).permute(0, 3, 2, 1, 4)
    return dict(codes=packed, scales=sw.contiguous().view(-1), s_dec=(1 / enc).reshape(1),
                rows=rows, cols=cols)


def _activations(g, *shape):
    """Gaussian values with a few large channels."""
    x = torch.randn(*shape, generator=g, device="cuda")
    return x * (1 + 9 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.01))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("fprop", "dgrad", "wgrad"):
        e = case["experts"]
        plan = _plan(_logits(case, g), case["top"])
        s["sizes"], s["offsets"] = plan["sizes"], plan["offsets"]
        s["largest"] = int(plan["sizes"].max())
        live = (plan["source"] >= 0).unsqueeze(1)
        rows = plan["source"].numel()
        if op == "wgrad":
            m, n = case["m"], case["n"]
            s["a"] = _quantised((_activations(g, rows, m) * live).t().contiguous())
            s["b"] = _quantised((_activations(g, rows, n) * live).t().contiguous())
            if case["fold"]:
                s["d"] = torch.randn(e, m, n, generator=g, device="cuda") * 30
        else:
            k, n = case["k"], case["n"]
            s["a"] = _quantised(_activations(g, rows, k) * live)
            shape = (e * n, k) if op == "fprop" else (n, e * k)
            s["b"] = _quantised(torch.randn(*shape, generator=g, device="cuda") * k ** -0.5)
    elif op == "norm":
        t, d = case["tokens"], case["d"]
        kind = torch.float32 if case["fp32"] else torch.bfloat16
        s["x"] = (_activations(g, t, d) * 2).to(kind)
        s["z"] = (_activations(g, t, d) * 0.3).bfloat16()
        s["w_post"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["w_pre"] = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["gate"] = None
        if case["gate"] != "none":
            shape = (d,) if case["gate"] == "channel" else (t, 1)
            s["gate"] = torch.rand(*shape, generator=g, device="cuda")
        if case["back"]:
            s["dy"] = torch.randn(t, d, generator=g, device="cuda").to(kind)
            s["dh"] = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    elif op == "route":
        t, e, top = case["tokens"], case["experts"], case["top"]
        x = _logits(case, g)
        masked = torch.rand(t, e, generator=g, device="cuda") < 0.05
        masked |= torch.rand(t, 1, generator=g, device="cuda") < 0.03  # padding tokens
        x = x.masked_fill(masked, -math.inf)
        s["logits"] = x if case["fp32"] else x.bfloat16()
        if case["back"]:
            s["dweight"] = torch.randn(t, top, generator=g, device="cuda")
    else:
        t, d, top = case["tokens"], case["d"], case["top"]
        s["plan"] = _plan(_logits(case, g), top)
        s["plan"]["weight"] = torch.softmax(torch.randn(t, top, generator=g, device="cuda"), 1)
        rows = s["plan"]["source"].numel()
        s["x"] = _activations(g, t, d).bfloat16()
        s["dy"] = torch.randn(t, d, generator=g, device="cuda").bfloat16()
        live = (s["plan"]["source"] >= 0).unsqueeze(1)
        s["out"] = (torch.randn(rows, d, generator=g, device="cuda") * live).bfloat16()
        s["dxe"] = (torch.randn(rows, d, generator=g, device="cuda") * live).bfloat16()
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from nvfp4_block_scaled_03_gb300 import binding as nv
    case = s["case"]
    op = case["op"]
    if op in ("fprop", "dgrad", "wgrad"):
        a = nv.operand(s["a"]["codes"], s["a"]["scales"], s["a"]["s_dec"], s["a"]["rows"],
                       s["a"]["cols"])
        b = s["b"]
        if op == "wgrad":
            b = nv.operand(b["codes"], b["scales"], b["s_dec"], b["rows"], b["cols"])
            mode = nv.D_F32_ACCUM if case["fold"] else nv.D_BF16
            return nv.nvfp4_group_wgrad(a, b, s["sizes"], s["offsets"], out=s.get("d"),
                                        d_mode=mode)
        if op == "fprop":
            b = nv.operand(b["codes"], b["scales"], b["s_dec"], b["rows"], b["cols"])
            return nv.nvfp4_group_gemm(a, b, s["sizes"], s["offsets"])
        b = nv.operand_t(b["codes"], b["scales"], b["s_dec"], b["cols"], b["rows"])
        return nv.nvfp4_group_gemm(a, b, s["sizes"], s["offsets"], b_view=1)
    if op == "norm":
        args = dict(w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], eps=EPS, x_scale=1.0,
                    z_scale=0.5)
        if case["back"]:
            return nv.nvfp4_residual_norm_bwd(s["dy"], s["dh"], s["x"], s["z"], **args)
        return nv.nvfp4_residual_norm_fwd(s["x"], s["z"], **args)
    if op == "route":
        mode = nv.ROUTE_CHOSEN if case["chosen"] else nv.ROUTE_ALL
        p = nv.nvfp4_route_fwd(s["logits"], case["top"], mode)
        got = dict(expert=p.expert, weight=p.weight, sizes=p.sizes, offsets=p.offsets, row=p.row,
                   source=p.source)
        if case["back"]:
            got["dlogits"] = nv.nvfp4_route_bwd(s["logits"], p, s["dweight"], mode)
        return got
    p = s["plan"]
    xe = nv.nvfp4_dispatch(s["x"], p["row"], p["source"])
    y = nv.nvfp4_combine(s["out"], p["row"], p["weight"])
    dout, dweight = nv.nvfp4_combine_bwd(s["dy"], s["out"], p["row"], p["source"], p["weight"])
    dx = nv.nvfp4_combine(s["dxe"], p["row"])
    return dict(xe=xe, y=y, dout=dout, dweight=dweight, dx=dx)


def _values(q):
    """The operand's values in 32 bits, without its decode scale."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                        device="cuda")
    rows, cols = q["rows"], q["cols"]
    c = torch.stack([q["codes"] & 15, q["codes"] >> 4], 2).view(rows, cols // 16, 16)
    s = q["scales"].view(rows // 128, cols // 64, 32, 4, 4).permute(0, 3, 2, 1, 4)
    s = s.reshape(rows, cols // 16).view(torch.float8_e4m3fn).float()
    return (grid[c.int()] * s.unsqueeze(2)).view(rows, cols)


def _grouped(s):
    """Index of each group's rows, padded to the largest group, and which count."""
    i = torch.arange(s["largest"], device="cuda")
    live = i < s["sizes"].unsqueeze(1)
    return torch.where(live, s["offsets"][:-1].unsqueeze(1) + i, 0), live


def _plain_product(s):
    case = s["case"]
    e, n, k = case["experts"], case["n"], case["k"]
    at, live = _grouped(s)
    a, b = _values(s["a"]), _values(s["b"])
    b = b.view(e, n, k) if case["op"] == "fprop" else b.view(n, e, k).transpose(0, 1)
    d = torch.bmm(a[at] * live.unsqueeze(2), b.transpose(1, 2)) * (s["a"]["s_dec"] * s["b"]["s_dec"])
    rows = s["a"]["rows"]
    out = torch.zeros(rows + 1, n, dtype=torch.bfloat16, device="cuda")
    out[torch.where(live, at, rows)] = d.bfloat16()
    return out[:rows]


def _plain_wgrad(s):
    at, live = _grouped(s)
    a = (_values(s["a"])[:, at] * live).transpose(0, 1)
    b = (_values(s["b"])[:, at] * live).permute(1, 2, 0)
    d = torch.bmm(a, b) * (s["a"]["s_dec"] * s["b"]["s_dec"])
    return s["d"].add_(d) if s["case"]["fold"] else d.bfloat16()


def _plain_norm(s):
    x, z = s["x"].float(), s["z"].float()
    g = 1.0 if s["gate"] is None else s["gate"]
    rz = torch.rsqrt(z.square().mean(1, keepdim=True) + EPS)
    zn = z * rz
    y = x + 0.5 * (g * (zn * s["w_post"]))
    ry = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    yn = y * ry
    if not s["case"]["back"]:
        return y.to(s["x"].dtype), (yn * s["w_pre"]).bfloat16()
    dy, dh = s["dy"].float(), s["dh"].float()
    dw_pre = (dh * yn).sum(0)
    u = dh * s["w_pre"]
    dy = dy + ry * (u - yn * (u * yn).mean(1, keepdim=True))
    q = 0.5 * dy
    dgate = None
    if s["gate"] is not None:
        dgate = q * zn * s["w_post"]
        dgate = dgate.sum(0) if s["case"]["gate"] == "channel" else dgate.sum(1, keepdim=True)
    dn = q * g
    dw_post = (dn * zn).sum(0)
    v = dn * s["w_post"]
    dz = rz * (v - zn * (v * zn).mean(1, keepdim=True))
    return dy.to(s["x"].dtype), dz.bfloat16(), dw_post, dgate, dw_pre


def _plain_route(s):
    case, x = s["case"], s["logits"].float()
    p = _plan(s["logits"], case["top"])
    some = p["expert"] >= 0
    at = p["expert"].clamp(min=0).long()
    top = x.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    ex = torch.exp(x - top)
    chosen = torch.where(some, ex.gather(1, at), 0.0)
    total = chosen.sum(1, keepdim=True) if case["chosen"] else ex.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    weight = chosen / total
    got = dict(p, weight=weight)
    if case["back"]:
        # w_i (dw_i - sum w dw), as differences: they stay exact where one weight is near 1
        dw = torch.where(some, s["dweight"], 0.0)
        apart = (weight.unsqueeze(1) * (dw.unsqueeze(2) - dw.unsqueeze(1))).sum(2)
        if case["chosen"]:
            dl = torch.zeros_like(x)
        else:
            others = ex.scatter_add(1, at, -chosen) / total
            apart = apart + others.sum(1, keepdim=True) * dw
            dl = -others * (weight * dw).sum(1, keepdim=True)
        dl.scatter_add_(1, at, weight * apart)
        got["dlogits"] = dl.to(s["logits"].dtype)
    return got


def _plain_move(s):
    p = s["plan"]
    t, top = p["row"].shape
    src = p["source"].long()
    live = (src >= 0).unsqueeze(1)
    token = src.clamp(min=0) // top
    row = p["row"].clamp(min=0).long()
    some = (p["row"] >= 0).unsqueeze(2)
    out, dy = s["out"], s["dy"].float()
    picked = torch.where(some, out[row].float(), 0.0)
    y = (picked * p["weight"].unsqueeze(2)).sum(1)
    w = p["weight"].reshape(-1)[src.clamp(min=0)].unsqueeze(1)
    return dict(xe=torch.where(live, s["x"][token], 0.0).bfloat16(), y=y.bfloat16(),
                dout=torch.where(live, w * dy[token], 0.0).bfloat16(),
                dweight=(picked * dy.unsqueeze(1)).sum(2),
                dx=torch.where(some, s["dxe"][row].float(), 0.0).sum(1).bfloat16())


_PLAIN = dict(fprop=_plain_product, dgrad=_plain_product, wgrad=_plain_wgrad, norm=_plain_norm,
              route=_plain_route, move=_plain_move)


# --------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------
def _decoded(q, rows, cols):
    """Rows and columns (slices) of an operand in 64 bits: nibble 2 i of a row
    is the low half of its byte i; the scale of row r, block c is the byte
    (r / 128, c / 4) * 512 + (r % 32) * 16 + (r / 32 % 4) * 4 + c % 4."""
    r = torch.arange(rows.start, rows.stop, device="cuda").unsqueeze(1)
    c = torch.arange(cols.start, cols.stop, device="cuda").unsqueeze(0)
    code = (q["codes"].view(-1)[r * (q["cols"] // 2) + c // 2].int() >> (4 * (c % 2))) & 15
    mag, exp = (code & 1).double(), (code >> 1) & 3
    value = torch.where(exp > 0, (1 + mag / 2) * torch.pow(2.0, (exp - 1).double()), mag / 2)
    value = torch.where(code >= 8, -value, value)
    b = c // 16
    byte = q["scales"][((r // 128) * (q["cols"] // 64) + b // 4) * 512 + (r % 32) * 16
                       + (r // 32 % 4) * 4 + b % 4].int()
    se, sm = byte >> 3, (byte & 7).double()
    scale = torch.where(se > 0, (1 + sm / 8) * torch.pow(2.0, (se - 7).double()),
                        sm / 8 * 2.0 ** -6)
    return value * scale


def _exact_product(s):
    case = s["case"]
    n, k = case["n"], case["k"]
    alpha = s["a"]["s_dec"].double() * s["b"]["s_dec"].double()
    out = torch.zeros(s["a"]["rows"], n, dtype=torch.float64, device="cuda")
    sizes, offsets = s["sizes"].tolist(), s["offsets"].tolist()
    for e, (size, first) in enumerate(zip(sizes, offsets)):
        if not size:
            continue
        a = _decoded(s["a"], slice(first, first + size), slice(0, k))
        for j in range(0, n, 2048):
            end = min(n, j + 2048)
            if case["op"] == "fprop":
                b = _decoded(s["b"], slice(e * n + j, e * n + end), slice(0, k))
            else:
                b = _decoded(s["b"], slice(j, end), slice(e * k, e * k + k))
            out[first:first + size, j:end] = a @ b.t() * alpha
    return out


def _exact_wgrad(s):
    case = s["case"]
    m, n = case["m"], case["n"]
    alpha = s["a"]["s_dec"].double() * s["b"]["s_dec"].double()
    out = torch.zeros(case["experts"], m, n, dtype=torch.float64, device="cuda")
    if case["fold"]:
        out += s["d"]
    for e, (size, first) in enumerate(zip(s["sizes"].tolist(), s["offsets"].tolist())):
        if size:
            cols = slice(first, first + size)
            out[e] += (_decoded(s["a"], slice(0, m), cols) @ _decoded(s["b"], slice(0, n), cols).t()
                       ) * alpha
    return out


def _exact_norm(s):
    """Forward from the formula; backward as the gradient that autograd gives of it."""
    back = s["case"]["back"]
    leaf = {k: s[k].double().requires_grad_(back) for k in ("x", "z", "w_post", "w_pre", "gate")
            if s[k] is not None}
    gate = leaf.get("gate", torch.ones((), dtype=torch.float64, device="cuda"))
    norm = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * w  # noqa: E731
    y = leaf["x"] + 0.5 * gate * norm(leaf["z"], leaf["w_post"])
    h = norm(y, leaf["w_pre"])
    if not back:
        return y, h
    torch.autograd.backward([y, h], [s["dy"].double(), s["dh"].double()])
    return tuple(leaf[k].grad if k in leaf else None
                 for k in ("x", "z", "w_post", "gate", "w_pre"))


def _exact_route(s):
    case = s["case"]
    x = s["logits"].double()
    none = x.amax(1, keepdim=True) == -math.inf
    p = torch.softmax(torch.where(none, 0.0, x), 1)
    # the slots' experts: the highest logits first, the lowest index among equals
    expert = torch.argsort(-x, dim=1, stable=True)[:, :case["top"]]
    live = torch.gather(x, 1, expert) > -math.inf
    if case["chosen"]:
        p = p * torch.zeros_like(p).scatter_(1, expert, 1.0)
        p = p / p.sum(1, keepdim=True)
    got = dict(weight=torch.where(live, torch.gather(p, 1, expert), 0.0))
    if case["back"]:
        # the softmax's Jacobian times the weights' gradient
        dp = torch.zeros_like(p).scatter_(1, expert, torch.where(live, s["dweight"].double(), 0.0))
        dl = p * (dp - (p * dp).sum(1, keepdim=True))
        got["dlogits"] = torch.where(none, 0.0, dl)
    return got


def _exact_move(s):
    p = s["plan"]
    t, top = p["row"].shape
    d = s["case"]["d"]
    dy = s["dy"].double()
    got = dict(xe=torch.zeros(p["source"].numel(), d, dtype=torch.float64, device="cuda"),
               y=torch.zeros(t, d, dtype=torch.float64, device="cuda"),
               dx=torch.zeros(t, d, dtype=torch.float64, device="cuda"),
               dweight=torch.zeros(t, top, dtype=torch.float64, device="cuda"))
    got["dout"] = torch.zeros_like(got["xe"])
    for j in range(top):
        there = torch.nonzero(p["row"][:, j] >= 0).squeeze(1)
        row = p["row"][there, j].long()
        w = p["weight"][there, j].double()[:, None]
        got["xe"][row] = s["x"][there].double()
        got["y"][there] += w * s["out"][row].double()
        got["dx"][there] += s["dxe"][row].double()
        got["dout"][row] = w * dy[there]
        got["dweight"][there, j] = (s["out"][row].double() * dy[there]).sum(1)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return dict(fprop=_exact_product, dgrad=_exact_product, wgrad=_exact_wgrad, norm=_exact_norm,
                route=_exact_route, move=_exact_move)[case["op"]](s)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, t = case["op"], case["tokens"]
    if op == "norm":
        wide = 4 if case["fp32"] else 2
        d = case["d"]
        side = d if case["gate"] == "channel" else t if case["gate"] == "row" else 0
        moved = (3 * wide + 3 * 2 if case["back"] else 2 * wide + 2 * 2) * t * d
        return dict(bytes=moved + 4 * (2 * d + side) * (2 if case["back"] else 1),
                    flops=(34 if case["back"] else 13) * t * d)
    e, top = case["experts"], case["top"]
    rows = t * top
    space = _rows_bound(rows, e)
    if op == "route":
        wide = 4 if case["fp32"] else 2
        out = rows * 12 + 4 * (2 * e + 1) + 4 * space
        return dict(bytes=t * e * wide * (2 if case["back"] else 1) + out + (4 * rows if case["back"] else 0),
                    flops=t * e * (5 if case["back"] else 3))
    if op == "move":
        d = case["d"]
        # x, dy, y, dx once each; the rows read (experts' outputs, gradients) and written (with padding)
        return dict(bytes=2 * d * (4 * t + 2 * rows + 2 * space) + 16 * rows + 4 * space,
                    flops=7 * rows * d)
    active = e * (1 - (1 - top / e) ** t)
    if op == "wgrad":
        m, n = case["m"], case["n"]
        d = 8 * active * m * n if case["fold"] else 2 * e * m * n
        return dict(bytes=rows * (m + n) * 0.5625 + d, flops=2 * rows * m * n)
    k, n = case["k"], case["n"]
    return dict(bytes=rows * k * 0.5625 + active * n * k * 0.5625 + space * n * 2,
                flops=2 * rows * n * k)
