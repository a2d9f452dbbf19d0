"""CPU oracle of scored routing and its gradient -- TEST INFRASTRUCTURE.

The definition in fp64 (numpy), sharing no code with the library:

    s_e   = 1 / (1 + exp(-l_e))   or   softmax(l)_e
    r_e   = s_e + b_e             or   l_e without a bias
    group = max r, or the sum of the two largest s + b, of E / G consecutive
            experts; only the experts of the best groups are candidates
    picks = the k best candidates by r; ties go to the lower index
    w_j   = scale s_j [/ sum of the chosen s]; an expert with b = -inf has s = 0 there
"""
from __future__ import annotations

import numpy as np


def scores(logits, score: str) -> np.ndarray:
    l = np.asarray(logits, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    e = np.exp(l - l.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def ranking(logits, bias, score: str, n_group: int, topk_group: int, group_top: int):
    """(rank [T, E] with -inf-or-lower entries as they are, candidate mask
    [T, E], group scores [T, G])."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores(l, score)
    both = s if bias is None else s + np.asarray(bias, np.float64)
    rank = l if bias is None else both
    size = E // n_group
    group = np.empty((T, n_group))
    for g in range(n_group):
        part = slice(g * size, (g + 1) * size)
        if group_top == 2:
            best = np.sort(both[:, part], axis=1)
            group[:, g] = best[:, -1] + best[:, -2]
        else:
            group[:, g] = rank[:, part].max(axis=1)
    mask = np.zeros((T, E), bool)
    for t in range(T):
        order = sorted(range(n_group), key=lambda g: (-group[t, g], g))
        for g in order[:topk_group]:
            mask[t, g * size:(g + 1) * size] = True
    return rank, mask, group


def choose(logits, k: int, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1):
    rank, mask, _ = ranking(logits, bias, score, n_group, topk_group, group_top)
    T, E = rank.shape
    idx = np.empty((T, k), np.int32)
    for t in range(T):
        cand = [e for e in range(E) if mask[t, e]]
        idx[t] = sorted(cand, key=lambda e: (-rank[t, e], e))[:k]
    return idx


def _chosen(logits, idx, bias, score):
    s = scores(logits, score)
    sel = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    if bias is not None:
        sel = np.where(np.asarray(bias)[idx] == -np.inf, 0.0, sel)
    return sel


def weights(logits, idx, bias=None, score="softmax", renormalize=True, scale=1.0):
    sel = _chosen(logits, idx, bias, score)
    if renormalize:
        total = sel.sum(axis=1, keepdims=True)
        sel = np.divide(sel, total, out=np.zeros_like(sel), where=total > 0)
    return scale * sel


def backward(dw, logits, idx, bias=None, score="softmax", renormalize=True, scale=1.0):
    """dL/dlogits for L = sum dw * weights(...), the choice held fixed."""
    dw = scale * np.asarray(dw, np.float64)
    s = scores(logits, score)
    sel = _chosen(logits, idx, bias, score)
    if renormalize:
        total = sel.sum(axis=1, keepdims=True)
        some = total > 0
        dsel = np.where(some, dw / np.where(some, total, 1.0), 0.0)
        dsel = dsel - (dsel * sel).sum(axis=1, keepdims=True) / np.where(some, total, 1.0)
    else:
        dsel = dw.copy()
    if bias is not None:
        dsel = np.where(np.asarray(bias)[idx] == -np.inf, 0.0, dsel)
    ds = np.zeros_like(s)
    np.put_along_axis(ds, idx.astype(np.int64), dsel, axis=1)
    if score == "sigmoid":
        return ds * s * (1.0 - s)
    if renormalize:   # the sum below is exactly zero: the common factor cancels
        return s * ds
    return s * (ds - (ds * s).sum(axis=1, keepdims=True))
