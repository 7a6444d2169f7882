"""Oracle of the scored router: scores, balance bias, groups of experts, gates, and their gradient, one
token at a time in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import math

import numpy as np

FLOAT_MAX = float(np.finfo(np.float32).max)


def scores(l, score):
    """(clean logits, scores) of one token's logits: NaN counts as -inf, +inf as the largest float."""
    l = np.array([-math.inf if math.isnan(v) else min(float(v), FLOAT_MAX) for v in l])
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return l, 1.0 / (1.0 + np.exp(-l))
    m = l.max()
    if m == -math.inf:
        return l, np.zeros_like(l)
    e = np.exp(l - m)
    return l, e / e.sum()


def route(logits, k, score="sigmoid", bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """(topk_idx [T, k], topk_gate [T, k] float64, scores [T, E] float64)."""
    T, E = logits.shape
    per = E // n_group
    idx = np.empty((T, k), np.int64)
    gate = np.empty((T, k))
    all_scores = np.empty((T, E))
    for t in range(T):
        l, s = scores(logits[t], score)
        c = [-math.inf if l[e] == -math.inf else s[e] + (0.0 if bias is None else float(bias[e])) for e in range(E)]
        c = [-math.inf if math.isnan(v) else v for v in c]
        rank = list(l) if bias is None else c
        value = []
        for g in range(n_group):
            best = sorted((v for v in c[g * per:(g + 1) * per] if v != -math.inf), reverse=True)[:group_top]
            value.append(sum(best) if best else -math.inf)
        kept = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
        inside = [e for e in range(E) if e // per in kept]
        chosen = sorted(inside, key=lambda e: (-rank[e], e))[:k]
        w = s[chosen]
        if renormalize and score == "softmax":      # the sum over all experts cancels
            w = scores(l[chosen], score)[1]
        elif renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        idx[t], gate[t], all_scores[t] = chosen, w * scale, s
    return idx, gate, all_scores


def route_bwd(logits, topk_idx, d_gate, score="sigmoid", renormalize=True, scale=1.0):
    """d_logits [T, E] from the Jacobian of the gates, the choice held fixed."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l, s = scores(logits[t], score)
        # Jacobian of the scores at the logits
        J = np.diag(s * (1.0 - s)) if score == "sigmoid" else np.diag(s) - np.outer(s, s)
        ds = np.zeros(E)
        w = s[topk_idx[t]]
        total = w.sum()
        for j, e in enumerate(topk_idx[t]):
            if not renormalize:
                ds[e] += scale * d_gate[t, j]
            elif total > 0:
                ds[e] += scale * (d_gate[t, j] - (w * d_gate[t]).sum() / total) / total
        out[t] = J @ ds
    return out
