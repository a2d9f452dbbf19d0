"""CPU oracle of what a training step runs around the layer -- TEST INFRASTRUCTURE.

Layer norm, the experts' balance loss and an AdamW step in fp64 (numpy), each with
what the tests need to bound its rounding; it shares no code with the library.

    y = (h - mean) / sqrt(var + eps) w + b
    loss = alpha / S sum_s sum_e (E c_se / (k n_s)) (sum_t p_te / n_s)
    m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
    p = p - lr (decay p + m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps))
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ layer norm
def norm(h, weight, bias, eps: float):
    """(y, mean, rstd)."""
    h = np.asarray(h, np.float64)
    mean = h.mean(axis=1, keepdims=True)
    var = np.square(h - mean).mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (h - mean) * rstd * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean[:, 0], rstd[:, 0]


def norm_backward(dy, h, mean, rstd, weight, dh=None):
    """(dx, dweight, dbias)."""
    dy, h, w = (np.asarray(a, np.float64) for a in (dy, h, weight))
    r = np.asarray(rstd, np.float64)[:, None]
    x = (h - np.asarray(mean, np.float64)[:, None]) * r
    g = dy * w
    dx = r * (g - g.mean(axis=1, keepdims=True) - x * (g * x).mean(axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * x).sum(axis=0), dy.sum(axis=0)


# ---------------------------------------------------------------- balance loss
def probabilities(logits, score: str):
    l = np.asarray(logits, np.float64)
    if score == "sigmoid":
        # of s = 1 / (1 + exp(-l)) only ratios count: exp(l - top) / (1 + exp(l)) exp(top)
        s = np.exp(-np.logaddexp(0.0, -l) + np.logaddexp(0.0, -l.max(axis=1, keepdims=True)))
    else:
        s = np.exp(l - l.max(axis=1, keepdims=True))
    return s / s.sum(axis=1, keepdims=True)


def members(T: int, seq_offsets=None, mask=None):
    """Row numbers of each sequence's counted tokens."""
    offsets = [0, T] if seq_offsets is None else [int(o) for o in seq_offsets]
    on = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    return [np.array([t for t in range(a, b) if on[t]], np.int64)
            for a, b in zip(offsets, offsets[1:])]


def balance(logits, topk_idx, alpha: float, score: str, seq_offsets=None, mask=None):
    """(loss, counts [S, E], tokens [S])."""
    l, idx = np.asarray(logits, np.float64), np.asarray(topk_idx)
    T, E = l.shape
    k = idx.shape[1]
    seqs = members(T, seq_offsets, mask)
    counts = np.zeros((len(seqs), E), np.int64)
    loss = 0.0
    for s, rows in enumerate(seqs):
        for t in rows:
            for e in idx[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if len(rows):
            mass = probabilities(l[rows], score).sum(axis=0)
            n = len(rows)
            loss += (E * counts[s] / (k * n) * (mass / n)).sum()
    return alpha / len(seqs) * loss, counts, np.array([len(r) for r in seqs])


def balance_backward(dloss: float, logits, counts, k: int, alpha: float, score: str,
                     seq_offsets=None, mask=None):
    """(dlogits, the sum of the absolute terms of each of its elements, the loads'
    means taken away)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    seqs = members(T, seq_offsets, mask)
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    for s, rows in enumerate(seqs):
        n = len(rows)
        if n == 0:
            continue
        f = dloss * alpha * E / (len(seqs) * k * float(n) ** 2)
        p = probabilities(l[rows], score)
        one = 1.0 if score == "softmax" else np.exp(-np.logaddexp(0.0, l[rows]))
        c = np.asarray(counts[s], np.float64)
        # sum p = 1: taken from all loads, a constant changes nothing but the rounding of
        # their difference, which is nothing where they are even
        c = c - k * n // E
        grad[rows] = f * p * one * (c - (p * c).sum(axis=1, keepdims=True))
        d = np.abs(c)
        size[rows] = abs(f) * p * one * (d + (p * d).sum(axis=1, keepdims=True))
    return grad, size


# ------------------------------------------------------------------------ AdamW
def adamw(p, g, m, v, t: int, lr, b1, b2, eps, decay, grad_scale=1.0):
    """(p, m, v) after step t."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    step = m / (1 - b1 ** t) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p - lr * (decay * p + step), m, v


E4M3 = sorted({s * (2.0 ** -9 * f if e == 0 else 2.0 ** (e - 7) * (1 + f / 8))
               for s in (-1, 1) for e in range(16) for f in range(8) if (e, f) != (15, 7)})


def e4m3_step(x):
    """The distance of e4m3's neighbours around |x| (at most 448)."""
    x = np.maximum(np.abs(np.asarray(x, np.float64)), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(x)) - 3)
