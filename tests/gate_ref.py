"""The gate in 64 bits with plain torch operations: what the tests of the gate compare with."""
import math

import torch


def scores(logits, score):
    l = logits.double()
    if score == "softmax":
        top = l.max(1, keepdim=True).values
        e = torch.exp(l - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
        return e / e.sum(1, keepdim=True).clamp(min=1e-300)
    return 1 / (1 + torch.exp(-l))


def choose(logits, bias, k, score, groups=1, top_groups=1, group_best=1):
    """(experts [T, k], which of them had a score [T, k])."""
    T, E = logits.shape
    s = scores(logits, score)
    order = logits.double() if bias is None else s + bias.double()
    c = s if bias is None else order
    ok = (logits > -math.inf) & ~torch.isnan(logits)
    if bias is not None:
        ok = ok & (bias > -math.inf)
    c, order = (torch.where(ok, v, torch.full_like(v, -math.inf)) for v in (c, order))
    if groups > 1:
        by = (order if group_best == 1 else c).reshape(T, groups, E // groups)
        top = torch.sort(by, dim=2, descending=True).values[..., :group_best]
        some = top[..., 0] > -math.inf
        gv = torch.where(top > -math.inf, top, torch.zeros_like(top)).sum(2)
        gv = torch.where(some, gv, torch.full_like(gv, -math.inf))
        best = torch.sort(gv, dim=1, descending=True, stable=True).indices[:, :top_groups]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=logits.device).scatter_(1, best, True)
        ok = ok & keep.repeat_interleave(E // groups, 1)
        order = torch.where(ok, order, torch.full_like(order, -math.inf))
    idx = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    return idx, ok.gather(1, idx)


def weights(logits, idx, has, score, renormalise, scale):
    """From the logarithms of the scores, which do not underflow."""
    l = logits.double()
    ls = torch.log_softmax(l, 1) if score == "softmax" else torch.nn.functional.logsigmoid(l)
    ls = torch.where(has, ls.gather(1, idx), torch.full_like(idx, -math.inf, dtype=torch.float64))
    none = ~has.any(1, keepdim=True)
    w = torch.softmax(torch.where(none, torch.zeros_like(ls), ls), 1) if renormalise else torch.exp(ls)
    return scale * torch.where(has & ~none, w, torch.zeros_like(w))


def dispatch(idx, E):
    flat = idx.reshape(-1)
    slots = torch.sort(flat, stable=True).indices
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(slots.numel(), device=slots.device)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)])
    return counts, offsets, rows.reshape(idx.shape), slots


def gradient(logits, idx, has, d, score, renormalise, scale):
    """d_logits of sum(w * d) by autograd."""
    l = logits.double().clone().requires_grad_()
    safe = torch.where(torch.isfinite(l), l, torch.full_like(l, -1e300)) if not torch.isfinite(logits).all() else l
    w = weights_of(safe, idx, has, score, renormalise, scale)
    g, = torch.autograd.grad((w * d.double()).sum(), l)
    return torch.nan_to_num(g)


def weights_of(l, idx, has, score, renormalise, scale):
    ls = torch.log_softmax(l, 1) if score == "softmax" else torch.nn.functional.logsigmoid(l)
    ls = ls.gather(1, idx)
    if not renormalise:
        return scale * torch.exp(ls) * has
    ls = ls.masked_fill(~has, -1e300)
    return scale * torch.softmax(ls, 1) * has
