"""Plain 64-bit references of the selection from logits and its gradient (the rules of
include/moe.h, moe_select_opts), written row by row."""
import numpy as np
import torch


def keys(l, b, kind):
    """(key, score) of one row in float64; masked experts: key -inf, score 0."""
    l = np.asarray(l, np.float64)
    b = np.zeros_like(l) if b is None else np.asarray(b, np.float64)
    with np.errstate(all="ignore"):
        if kind == 0:
            key = l + b
            key = np.where(np.isnan(key), -np.inf, key)
            m = key.max()
            e = np.where(key == -np.inf, 0.0, np.where(key == m, 1.0, np.exp(key - m)))
            return key, (e / e.sum() if e.sum() > 0 else e)
        s = 1.0 / (1.0 + np.exp(-l))
        masked = np.isnan(l) | (l == -np.inf)
        s = np.where(masked, 0.0, s)
        key = np.where(masked, -np.inf, s + b)
        return np.where(np.isnan(key), -np.inf, key), s


def choose(key, k, groups, keep, top):
    """The chosen experts in order; and the smallest non-zero gap that a comparison hung on."""
    E = len(key)
    per = E // groups
    gap = np.inf
    allowed = np.ones(E, bool)
    if keep < groups:
        g = []
        for i in range(groups):
            v = sorted((x for x in key[i * per:(i + 1) * per] if x > -np.inf), reverse=True)
            g.append(sum(v[:top]) if v else -np.inf)
        order = sorted(range(groups), key=lambda i: (-g[i], i))
        a, c = g[order[keep - 1]], g[order[keep]]
        if a != c:
            gap = min(gap, a - c)
        for i in order[keep:]:
            allowed[i * per:(i + 1) * per] = False
    order = sorted((e for e in range(E) if allowed[e]), key=lambda e: (-key[e], e))
    for x, y in zip(order[:k], order[1:k + 1]):
        if key[x] != key[y]:
            gap = min(gap, key[x] - key[y])
    return order[:k], gap


def select(logits, bias, kind, k, groups=1, keep=1, top=1, renorm=True):
    """(idx [T, k], w [T, k], prob_sum [E], smallest gap) in float64."""
    T, E = logits.shape
    idx, w, prob, gap = np.zeros((T, k), np.int32), np.zeros((T, k)), np.zeros(E), np.inf
    for t in range(T):
        key, score = keys(logits[t], bias, kind)
        idx[t], g = choose(key, k, groups, keep, top)
        gap = min(gap, g)
        if score.sum() > 0:
            prob += score / score.sum()
        if renorm and kind == 0:  # relative to the best chosen key: no underflow
            ck = key[idx[t]]
            with np.errstate(all="ignore"):
                e = np.where(ck == -np.inf, 0.0, np.where(ck == ck[0], 1.0, np.exp(ck - ck[0])))
            w[t] = e / e.sum() if e.sum() > 0 else 0.0
        else:
            w[t] = score[idx[t]]
            if renorm:
                w[t] = w[t] / w[t].sum() if w[t].sum() > 0 else 0.0
    return idx, w, prob, gap


def loss(l, bias, kind, idx, renorm, d_w, d_prob):
    """sum d_w w + sum d_prob prob_sum as a differentiable float64 torch scalar (no masks)."""
    if kind == 0:
        score = q = torch.softmax(l if bias is None else l + bias, dim=1)
    else:
        score = torch.sigmoid(l)
        q = score / score.sum(1, keepdim=True)
    w = score.gather(1, idx.long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    out = (w * d_w).sum()
    return out if d_prob is None else out + (q.sum(0) * d_prob).sum()
