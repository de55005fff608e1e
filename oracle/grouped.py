"""Plain float64 definitions of routing with groups and a bias, and of gradient clipping, in NumPy."""
from __future__ import annotations

import numpy as np


def _shares(x):
    """exp(x) over its sum, row by row; -inf has no share, and +infs have all of it in equal parts."""
    m = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(np.isneginf(x), 0.0, np.where(x == m, 1.0, np.exp(x - m)))
    s = e.sum(1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s != 0)


def scores(logits, score):
    """softmax over each row, or sigmoid; a softmax row of -inf alone scores 0 everywhere."""
    l = np.asarray(logits, np.float64)
    if score == "softmax":
        return _shares(l)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-l))


def choose(logits, k, score, groups=1, topk_groups=1, group_top=2, bias=None):
    """[T, k] experts, one token and one pick at a time. A logit of -inf stays behind the others
    whatever its bias; groups whose sum such experts make -inf go by their best."""
    v = scores(logits, score)
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    elif groups == 1 or group_top == 1:  # nothing is added: by the logits, which do not saturate
        v = np.asarray(logits, np.float64)
    v = np.where(np.isneginf(logits), -np.inf, v)
    T, E = v.shape
    size = E // groups
    ids = np.empty((T, k), np.int64)
    for t in range(T):
        top = [sorted(v[t, g * size:(g + 1) * size])[::-1][:group_top] for g in range(groups)]
        best = [(sum(x), x[0] if sum(x) == -np.inf else 0.0) for x in top]
        stay = sorted(range(groups), key=lambda g: (-best[g][0], -best[g][1], g))[:topk_groups]
        free = [e for e in range(E) if e // size in stay]
        ids[t] = sorted(free, key=lambda e: (-v[t, e], e))[:k]
    return ids


def weights(logits, ids, score, renorm, scale):
    """Weights of the chosen. Renormalised: the ratios of the scores, from their logarithms."""
    l = np.take_along_axis(np.asarray(logits, np.float64), ids, 1)
    if not renorm:
        return scale * np.take_along_axis(scores(logits, score), ids, 1)
    return scale * _shares(-np.logaddexp(0.0, -l) if score == "sigmoid" else l)


def weights_backward(logits, ids, dw, score, renorm, scale):
    """d logits from the gradient of the weights."""
    l = np.asarray(logits, np.float64)
    dw = np.asarray(dw, np.float64)
    out = np.zeros_like(l)
    if renorm:
        p = weights(logits, ids, score, True, 1.0)
        d = scale * p * (dw - (dw * p).sum(1, keepdims=True))
        if score == "sigmoid":
            d = d * scores(-np.take_along_axis(l, ids, 1), "sigmoid")
        np.put_along_axis(out, ids, d, 1)
        return out
    s = scores(l, score)
    np.put_along_axis(out, ids, scale * dw, 1)
    if score == "sigmoid":
        return out * s * scores(-l, "sigmoid")
    return s * (out - (out * s).sum(1, keepdims=True))


def clip(grads, max_norm, eps=1e-6):
    """(norm, the gradients scaled to at most max_norm)."""
    norm = np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads))
    c = min(1.0, max_norm / (norm + eps))
    return norm, [np.asarray(g, np.float64) * c for g in grads]
