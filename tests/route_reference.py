"""The router, its balance loss and their gradient from their definitions in 64
bits, with error bounds of a computation in fp32.

Bounds.  u = 2^-24.  exp of a difference of logits, rounded, is off by u times
the difference besides 2 units of its last place; with R the largest
difference that matters (from the row's largest logit, or of a sigmoid's
logit from 0) a score is good to (R + 8) 2 u of itself, a sum of E scores,
all positive, in any order of at most E / 32 + 8 additions a term, to
(R + E / 32 + 16) 2 u.  `relative` adds both for a ratio and a product or
two.  An output rounded to b bits is off by half a step besides,
torch.finfo(type).eps / 2 of it, or half the least subnormal.
"""
import math

import torch

U = 2.0 ** -24


def relative(l):
    """Relative error of a normalised score of logits l (64 bits), for each row; -inf and NaN aside."""
    ok = torch.isfinite(l)
    top = torch.where(ok, l, -math.inf).amax(1, keepdim=True)
    spread = torch.where(ok, torch.maximum((top - l).abs(), l.abs()), 0.0).amax(1)
    return (2 * spread + l.shape[1] / 16 + 64) * 2 * U


def scores(l, score):
    """(s, p): scores, and over their sum."""
    if score == "softmax":
        s = torch.softmax(l, 1)
        return s, s
    s = torch.sigmoid(l)
    return s, torch.softmax(torch.nn.functional.logsigmoid(l), 1)


def ordered(key, n):
    """The n largest of each row: NaN above all, equal ones by the lower index (torch's stable sort)."""
    return torch.sort(key + 0.0, dim=1, descending=True, stable=True).indices[:, :n]


def route(l, K, score, bias=None, mask=None, groups=1, topk_groups=1, normalize=True, scale=1.0):
    """topk_idx and topk_weights from logits in 64 bits."""
    l = l.double()
    T, E = l.shape
    s = scores(l, score)[0]
    c = s if bias is None else s + bias.double()
    c = torch.where(l == -math.inf, -math.inf, c)
    if topk_groups < groups:
        g = c.reshape(T, groups, E // groups)
        two = torch.sort(g, dim=2, descending=True).values[:, :, :2]
        best = two[:, :, 0]
        if two.shape[2] > 1:
            best = best + torch.where(two[:, :, 1] == -math.inf, 0.0, two[:, :, 1])
        keep = torch.zeros((T, groups), dtype=torch.bool, device=l.device)
        keep.scatter_(1, ordered(best, topk_groups), True)
        c = torch.where(keep.repeat_interleave(E // groups, 1), c, -math.inf)
    key = c if bias is not None else torch.where(c == -math.inf, -math.inf, l)
    idx = ordered(key, K)
    there = key.gather(1, idx) != -math.inf
    if mask is not None:
        there &= mask.bool()[:, None]
    chosen = l.gather(1, idx)
    if normalize:
        v = torch.where(there, chosen if score == "softmax" else torch.nn.functional.logsigmoid(chosen), -math.inf)
        w = torch.softmax(v, 1) * scale
    else:
        w = s.gather(1, idx) * scale
    return torch.where(there, idx, -1), torch.where(there, w, 0.0)


def sequence_of(T, offset, device):
    """Sequence of every token; -1 where there is none."""
    if offset is None:
        return torch.zeros(T, dtype=torch.int64, device=device)
    q = torch.full((T,), -1, dtype=torch.int64, device=device)
    for i, (a, b) in enumerate(zip(offset.tolist(), offset.tolist()[1:])):
        q[a:b] = i
    return q


def takes_part(l, mask):
    live = (l != -math.inf).any(1)
    return live if mask is None else live & mask.bool()


def balance(l, idx, score, offset=None, mask=None, coeff=1.0):
    """loss, load and counts in 64 bits."""
    l = l.double()
    T, E = l.shape
    K = idx.shape[1]
    S = 1 if offset is None else offset.numel() - 1
    q = torch.where(takes_part(l, mask), sequence_of(T, offset, l.device), -1)
    p = scores(l, score)[1]
    loss, load = 0.0, torch.zeros((S, E), dtype=torch.float64, device=l.device)
    counts = torch.zeros((S, E), dtype=torch.int64, device=l.device)
    for i in range(S):
        at = q == i
        n = int(at.sum())
        if n == 0:
            continue
        named = idx[at].reshape(-1)
        counts[i] = torch.bincount(named[(named >= 0) & (named < E)], minlength=E)
        load[i] = coeff / S * counts[i].double() * E / (K * n) / n
        loss = loss + (load[i] * p[at].sum(0)).sum()
    return loss, load, counts


def backward(l, idx, score, d_weights=None, load=None, d_loss=None, offset=None, mask=None, normalize=True, scale=1.0):
    """(d_logits, bound before the output's rounding) by the formulas, in 64 bits."""
    l = l.double()
    T, E = l.shape
    s, p = scores(l, score)
    live = takes_part(l, mask)
    p = torch.where(live[:, None], p, 0.0)
    s = torch.where(live[:, None], s, 0.0)
    out, big = torch.zeros_like(l), torch.zeros_like(l)
    outer = torch.ones_like(l) if score == "softmax" else torch.sigmoid(-l)
    if load is not None:
        q = sequence_of(T, offset, l.device)
        a = torch.where((q >= 0)[:, None], load.double()[q.clamp_min(0)], 0.0) * d_loss.double()
        out += outer * p * (a - (a * p).sum(1, keepdim=True))
        big += outer * p * (a.abs() + (a.abs() * p).sum(1, keepdim=True))
    if d_weights is not None:
        there = (idx >= 0) & (idx < E) & live[:, None]
        at = torch.where(there, idx, 0)
        g = torch.where(there, d_weights.double() * scale, 0.0)
        chosen = l.gather(1, at)
        if normalize:
            v = torch.where(there, chosen if score == "softmax" else torch.nn.functional.logsigmoid(chosen), -math.inf)
            w = torch.where(there & (v != -math.inf).any(1, keepdim=True), torch.softmax(v, 1), 0.0)
            r, rb = w * (g - (g * w).sum(1, keepdim=True)), w * (g.abs() + (g.abs() * w).sum(1, keepdim=True))
        else:
            r = torch.where(there, s.gather(1, at), 0.0) * g
            rb = r.abs()
            if score == "softmax":
                out -= p * r.sum(1, keepdim=True)
                big += p * rb.sum(1, keepdim=True)
        if score == "sigmoid":
            r, rb = r * torch.sigmoid(-chosen), rb * torch.sigmoid(-chosen)
        out.scatter_add_(1, at, torch.where(there, r, 0.0))
        big.scatter_add_(1, at, torch.where(there, rb, 0.0))
    zero = ~live[:, None]
    return torch.where(zero, 0.0, out), torch.where(zero, 0.0, big) * 2 * relative(l)[:, None]


def rounded(value, bound, dtype):
    """The bound after rounding to dtype."""
    info = torch.finfo(dtype)
    return bound + info.eps / 2 * (value.abs() + bound) + info.smallest_normal * info.eps
