"""Plain 64-bit forms of the mixture-of-experts operators, from their formulas
(NumPy only), with the magnitudes that the tolerances of the tests scale with.

Tolerances.  The kernels work in FP32 and round once to the output's type.  A
value s = sum of n terms taken in FP32 by any order of partial sums of at most
r additions in a row is off by at most r 2^-24 sum|terms| (to first order).
The norms add at most 16 * 8 products in a thread, 5 across a warp and 16
across warps: r = 149, and a mean of squares enters through its square root
(half the relative error); the few further roundings of a formula add less
than 2^-20 relative.  E_NORM = 2^-16 covers their sum with room for a term that
meets two such means.  A bf16 output adds half a unit in the last place.
"""
import numpy as np

E_NORM = 2.0 ** -16


def bf16(a):
    """Round to the nearest bf16 (ties to even), as float64."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    r = (u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)
    return r.view(np.float32).astype(np.float64)


def half_ulp_bf16(v):
    a = np.abs(v)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    return np.where(a > 0, np.maximum(2.0 ** (e - 8), 2.0 ** -134), 0.0)


def norm_fwd(x, z, w_post, gate, w_pre, eps, a, b):
    """y, h and the sizes of their terms (|a x| + |b g n|, and that through the norm)."""
    y, my = a * x, np.abs(a * x)
    if z is not None:
        n = z / np.sqrt((z * z).mean(1, keepdims=True) + eps) * w_post
        t = b * (n if gate is None else gate * n)
        y, my = y + t, my + np.abs(t)
    if w_pre is None:
        return y, None, my, None
    ry = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    return y, y * ry * w_pre, my, (my + np.abs(y)) * ry * np.abs(w_pre)


def norm_bwd(dy, dh, x, z, w_post, gate, w_pre, eps, a, b):
    """{name: (gradient, size of its terms)}."""
    out = {}
    y, _, my, _ = norm_fwd(x, z, w_post, gate, w_pre, eps, a, b)
    d = np.zeros_like(x) if dy is None else dy
    md = np.abs(d)
    if w_pre is not None:
        ry = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        yh, u = y * ry, dh * w_pre
        myh = my * ry
        out["dw_pre"] = (dh * yh).sum(0), (np.abs(dh) * myh).sum(0)
        d = d + ry * (u - yh * (u * yh).mean(1, keepdims=True))
        md = md + ry * (np.abs(u) + 2 * myh * (np.abs(u) * myh).mean(1, keepdims=True))
    out["dx"] = a * d, np.abs(a) * md
    if z is not None:
        rz = 1 / np.sqrt((z * z).mean(1, keepdims=True) + eps)
        zh = z * rz
        q, mq = b * d, np.abs(b) * md
        g = 1.0 if gate is None else gate
        if gate is not None:
            t, mt = q * zh * w_post, mq * np.abs(zh * w_post)
            row = gate.ndim == 2
            out["dgate"] = ((t.sum(1, keepdims=True), mt.sum(1, keepdims=True)) if row
                            else (t.sum(0), mt.sum(0)))
        dn, mdn = q * g, mq * np.abs(g)
        out["dw_post"] = (dn * zh).sum(0), (mdn * np.abs(zh)).sum(0)
        v, mv = dn * w_post, mdn * np.abs(w_post)
        out["dz"] = (rz * (v - zh * (v * zh).mean(1, keepdims=True)),
                     rz * (mv + np.abs(zh) * (mv * np.abs(zh)).mean(1, keepdims=True)))
    return out


def route(logits, top, chosen):
    """expert, weight (64 bits) and the plan of float32 logits [T, E]."""
    T, E = logits.shape
    x = logits.astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    order = np.argsort(-x, axis=1, kind="stable")[:, :top]
    live = np.take_along_axis(x, order, 1) > -np.inf
    expert = np.where(live, order, -1)
    m = x.max(1, keepdims=True)
    m = np.where(m > -np.inf, m, 0.0)
    p = np.exp(x - m)
    c = np.where(live, np.take_along_axis(p, order, 1), 0.0)
    total = c.sum(1, keepdims=True) if chosen else p.sum(1, keepdims=True)
    weight = c / np.where(total > 0, total, 1.0)
    sizes = np.array([(expert == e).sum() for e in range(E)], dtype=np.int64)
    offsets = np.concatenate([[0], np.cumsum((sizes + 127) // 128 * 128)])
    n = T * top
    rows = (n + 127 * min(E, n)) // 128 * 128
    row = np.full(n, -1, dtype=np.int64)
    source = np.full(rows, -1, dtype=np.int64)
    taken = offsets[:-1].copy()
    for i, e in enumerate(expert.reshape(-1)):
        if e >= 0:
            row[i], source[taken[e]] = taken[e], i
            taken[e] += 1
    return dict(expert=expert, weight=weight, sizes=sizes, offsets=offsets,
                row=row.reshape(T, top), source=source, p=p / np.where(p.sum(1, keepdims=True) > 0,
                                                                      p.sum(1, keepdims=True), 1))


def route_bwd(r, dweight, chosen):
    """dlogits and the size of its terms, from route()'s answer."""
    T, E = r["p"].shape
    live = r["expert"] >= 0
    w, dw = r["weight"], np.where(live, dweight, 0.0)
    dp = np.zeros((T, E))
    t = np.arange(T)[:, None]
    at = np.where(live, r["expert"], 0)
    np.add.at(dp, (t, at), np.where(live, dw, 0.0))
    if chosen:
        p = np.zeros((T, E))
        np.add.at(p, (t, at), np.where(live, w, 0.0))
    else:
        p = r["p"]
    mean = (p * dp).sum(1, keepdims=True)
    return p * (dp - mean), p * (np.abs(dp) + (p * np.abs(dp)).sum(1, keepdims=True))


GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])


def decode(codes, scales_sw, s_dec, rows, cols):
    """Values (64 bits) of a K-major operand from its bytes."""
    c = codes.reshape(rows, cols // 2)
    v = np.empty((rows, cols))
    v[:, 0::2], v[:, 1::2] = GRID[c & 15], GRID[c >> 4]
    r = np.arange(rows)[:, None]
    k = np.arange(cols // 16)[None, :]
    kg = (cols // 16 + 3) // 4
    b = scales_sw[((r // 128) * kg + k // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4]
    e, m = (b >> 3).astype(np.int64), (b & 7).astype(np.float64)
    s = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)
    return v * np.repeat(s, 16, axis=1) * float(s_dec)
