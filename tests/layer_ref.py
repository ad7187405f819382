"""Plain 64-bit forms of the steps around the expert products, for the GPU
tests: numpy, from the formulas in include/moe_layer.h, nothing shared with
the library."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24                                  # half a step of fp32 around 1
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def softmax(l: np.ndarray) -> np.ndarray:
    """Rows with every entry -inf are 0, not 0/0."""
    top = l.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.exp(l - np.where(top == -np.inf, 0.0, top))
        s = e.sum(axis=1, keepdims=True)
        return np.where(s == 0.0, 0.0, e / np.where(s == 0.0, 1.0, s))


def choice(l: np.ndarray, topk: int) -> np.ndarray:
    """The topk largest of each row, NaN above +inf, the lower index first."""
    T, E = l.shape
    key = np.where(np.isnan(l), 0.0, l)
    index = np.broadcast_to(np.arange(E), l.shape)
    return np.lexsort((index, -key, ~np.isnan(l)), axis=1)[:, :topk]


def route(l, topk, renorm, scale=1.0):
    p = softmax(l)
    ids = choice(l, topk)
    w = np.take_along_axis(p, ids, 1)
    if renorm:
        s = w.sum(axis=1, keepdims=True)
        w = np.where(s == 0.0, 0.0, w / np.where(s == 0.0, 1.0, s))
    return ids, scale * w


def balance(l, ids, off, coef):
    S, (T, E), K = len(off) - 1, l.shape, ids.shape[1]
    p = softmax(l)
    counts, probs, loss = np.zeros((S, E), np.int64), np.zeros((S, E)), 0.0
    for s in range(S):
        for t in range(off[s], off[s + 1]):
            for e in ids[t]:
                counts[s, e] += l[t, e] != -np.inf
        n = off[s + 1] - off[s]
        if n:
            probs[s] = p[off[s]:off[s + 1]].mean(axis=0)
            loss += coef / S * (counts[s] * E / (K * n) * probs[s]).sum()
    return counts, probs, loss


def balance_only(l, ids, off, coef, counts):
    """The loss as a function of the logits, counts held (for differences)."""
    S, E, K = len(off) - 1, l.shape[1], ids.shape[1]
    p = softmax(l)
    return sum(coef / S * (counts[s] * E / (K * (off[s + 1] - off[s])) * p[off[s]:off[s + 1]].mean(axis=0)).sum()
               for s in range(S) if off[s + 1] > off[s])


def route_backward(l, ids, dw, renorm, scale=1.0, off=None, coef=0.0, counts=None, dloss=1.0):
    """-> (dlogits, the sum of the magnitudes that make it up, for error bounds)."""
    T, E = l.shape
    K = ids.shape[1]
    p = softmax(l)
    c = np.zeros((T, E))
    if off is not None:
        S = len(off) - 1
        for s in range(S):
            n = off[s + 1] - off[s]
            if n:
                c[off[s]:off[s + 1]] = dloss * coef * E * counts[s] / (S * K * float(n) ** 2)
    d = p * (c - (p * c).sum(axis=1, keepdims=True))
    size = p * (np.abs(c) + (p * np.abs(c)).sum(axis=1, keepdims=True))
    if dw is None:
        return d, size
    rows = np.arange(T)
    pick = np.take_along_axis(p, ids, 1)
    if renorm:
        s = pick.sum(axis=1, keepdims=True)
        q = np.where(s == 0.0, 0.0, pick / np.where(s == 0.0, 1.0, s))
        add = scale * q * (dw - (q * dw).sum(axis=1, keepdims=True))
        mag = abs(scale) * q * (np.abs(dw) + (q * np.abs(dw)).sum(axis=1, keepdims=True))
    else:
        add = scale * pick * dw
        mag = np.abs(add)
        d = d - p * add.sum(axis=1, keepdims=True)
        size = size + p * mag.sum(axis=1, keepdims=True)
    for k in range(K):
        d[rows, ids[:, k]] += add[:, k]
        size[rows, ids[:, k]] += mag[:, k]
    return d, size


def adapters(x, base, ids, a, b, scale, ranks):
    """-> (out, the update, sum of the magnitudes of the update's terms)."""
    out, size = base.copy(), np.zeros_like(base)
    for t, i in enumerate(ids):
        if 0 <= i < a.shape[0]:
            r = min(max(int(ranks[i]), 0), a.shape[1])
            out[t] += scale[i] * (b[i][:, :r] @ (a[i][:r] @ x[t]))
            size[t] = abs(scale[i]) * (np.abs(b[i][:, :r]) @ (np.abs(a[i][:r]) @ np.abs(x[t])))
    return out, out - base, size
