"""Scored routing in 64 bits, from its definition (torch, any device)."""
import math

import torch


def scores(logits, score):
    """(scores, which are open) in 64 bits."""
    top = torch.finfo(logits.dtype).max
    open_ = logits > -math.inf
    x = torch.where(open_, logits.double().clamp(max=top), 0.0)
    if score == 1:
        s = torch.sigmoid(x)
    else:
        most = torch.where(open_, x, -1e300).amax(1, keepdim=True)
        e = torch.where(open_, torch.exp(x - most), 0.0)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(open_, s, 0.0), open_, x


def choose(logits, top, score, bias=None, groups=1, kept=None, group_top=2):
    """The chosen experts [tokens, top], -1 for none."""
    s, open_, x = scores(logits, score)
    t, e = s.shape
    key = x if bias is None else s + bias.double()
    worth_of = s if bias is None else key
    if bias is None and group_top == 1:
        worth_of = x
    ninf = torch.full_like(key, -math.inf)
    key = torch.where(open_, key, ninf)
    if groups > 1:
        v = torch.where(open_, worth_of, ninf).view(t, groups, -1)
        best = torch.sort(v, dim=2, descending=True).values[:, :, :group_top]
        live = best[:, :, 0] > -math.inf
        worth = torch.where(best > -math.inf, best, 0.0).sum(2)
        worth = torch.where(live, worth, -math.inf)
        order = torch.argsort(worth, dim=1, descending=True, stable=True)
        keep = torch.zeros_like(worth, dtype=torch.bool)
        keep.scatter_(1, order[:, :groups if kept is None else kept], True)
        key = torch.where(keep.repeat_interleave(e // groups, 1), key, ninf)
    value, index = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(value[:, :top] > -math.inf, index[:, :top], -1)


def weights(logits, expert, score, renormalise, scale):
    """Weights of given experts, differentiable in the logits; a chosen sigmoid's
    share of its row is taken as e^(log s_i - log s_max)."""
    some = expert >= 0
    at = expert.clamp(min=0)
    if score == 1:
        log_s = torch.nn.functional.logsigmoid(logits.gather(1, at))
    else:
        log_s = torch.log_softmax(logits, 1).gather(1, at)
    if not renormalise:
        return torch.where(some, scale * torch.exp(log_s), 0.0)
    log_s = torch.where(some, log_s, -1e300)
    w = torch.softmax(log_s, 1)
    return torch.where(some, scale * w, 0.0)


def plan(expert, experts, rows):
    """sizes, offsets, row and source of a choice, slot by slot."""
    t, top = expert.shape
    flat = expert.reshape(-1).tolist()
    sizes = [0] * experts
    for e in flat:
        if e >= 0:
            sizes[e] += 1
    offsets = [0]
    for n in sizes:
        offsets.append(offsets[-1] + (n + 127) // 128 * 128)
    nxt, row, source = list(offsets), [], [-1] * rows
    for i, e in enumerate(flat):
        if e < 0:
            row.append(-1)
            continue
        row.append(nxt[e])
        source[nxt[e]] = i
        nxt[e] += 1
    return sizes, offsets, row, source
