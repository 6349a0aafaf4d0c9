"""A model's gate and the norms around the MoE block, plainly (oracle; test infrastructure only).

gate     scores s = softmax(l) or sigmoid(l); choice c = s + balance bias; the experts of the groups of
         largest value (sum of a group's `group_top` largest choices); the k largest choices, equal
         choices to the lower expert; weights s (/ sum over the chosen) * scale.  Without a balance bias
         the choice is ordered as the logits.  NaN or -inf logits, and NaN or -inf balance biases, take an
         expert out; slots without an expert hold -1 and weight 0.
norm     z / sqrt(mean(z^2) + eps) * weight.

fp64 throughout.
"""
from __future__ import annotations

import numpy as np


def _scores(l, score):
    """fp64 scores of fp64 logits (NaN already replaced by -inf)."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(1, keepdims=True)
        z = np.where(l == m, 1.0, np.exp(l - m))
        z[~(l > -np.inf)] = 0.0
        return z / z.sum(1, keepdims=True)


def gate(logits, k, score="softmax", balance=None, n_groups=1, topk_groups=1, group_top=1, renormalize=True,
         scale=1.0):
    """(idx [T,k] int32, w [T,k] fp64) of fp32 logits [T,E]."""
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    T, E = l.shape
    s = _scores(l, score)
    b = np.zeros(E) if balance is None else np.asarray(balance, np.float64)
    live = (l > -np.inf) & (b > -np.inf)[None, :]
    c = np.where(live, s + np.where(b > -np.inf, b, 0.0)[None, :], -np.inf)
    order = np.where(live, l, -np.inf) if balance is None else c
    gs = E // n_groups
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        ok = live[t].copy()
        if topk_groups < n_groups:
            by = order if group_top == 1 else c
            value = []
            for g in range(n_groups):
                top = sorted((v for v in by[t, g * gs:(g + 1) * gs] if v > -np.inf), reverse=True)[:group_top]
                value.append(sum(top) if top else -np.inf)
            kept = sorted(range(n_groups), key=lambda g: (-value[g], g))[:topk_groups]
            for g in range(n_groups):
                if g not in kept:
                    ok[g * gs:(g + 1) * gs] = False
        cand = sorted(np.nonzero(ok)[0], key=lambda e: (-order[t, e], e))[:k]
        n = len(cand)
        idx[t, :n] = cand
        if n == 0:
            continue
        x = l[t, cand]
        with np.errstate(over="ignore", invalid="ignore"):
            if not renormalize:
                v = s[t, cand]
            elif score == "softmax":
                v = np.where(x == x.max(), 1.0, np.exp(x - x.max()))
                v = v / v.sum()
            else:                              # log sigmoid(x) = min(x, 0) - log(1 + e^-|x|), shifted by its largest part
                f = np.minimum(x, 0.0)
                v = np.where(f == f.max(), 1.0, np.exp(f - f.max())) / (1.0 + np.exp(-np.abs(x)))
                v = v / v.sum()
        w[t, :n] = v * scale
    return idx, w


def rmsnorm(z, weight, eps):
    z = np.asarray(z, np.float64)
    with np.errstate(all="ignore"):
        return z / np.sqrt((z * z).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)[None, :]


def combine(y_perm, inv_perm, topk_w, shared):
    """(sum, sum of the terms' magnitudes): the weighted unpermute, dropped slots left out."""
    y = np.asarray(y_perm, np.float64)
    T, k = inv_perm.shape
    z = np.zeros((T, y.shape[1]))
    mag = np.zeros_like(z)
    for t in range(T):
        for j in range(k):
            r = int(inv_perm[t, j])
            if 0 <= r < len(y):
                term = np.float64(topk_w[t, j]) * y[r]
                z[t] += term
                mag[t] += np.abs(term)
        if shared:
            z[t] += y[T * k + t]
            mag[t] += np.abs(y[T * k + t])
    return z, mag
