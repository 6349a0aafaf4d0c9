"""The load of a batch's experts as losses, and the gradient of a gate, plainly (oracle; test infrastructure only).

p        softmax(l), or sigmoid(l) / sum of sigmoids; logits of NaN and -inf take no part
balance  sum_e f_e * mean_t p_te, f_e = E / (k N) * (how often e was chosen), per sequence of N tokens
z        mean_t logsumexp(l_t)^2
weights  scale * score of the chosen, divided by their sum if renormalised

fp64 throughout.  The gradient is written from the formulas; tests hold it against differences of the losses.
"""
from __future__ import annotations

import numpy as np


def _parts(l, score):
    """(softmax, p, slope, lse) of fp64 logits [T,E] without NaN; slope is d log(score_i) / d l_i of a lone score."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        m = l.max(1, keepdims=True)
        e = np.where(l == m, 1.0, np.exp(l - m))
        e[~(l > -np.inf)] = 0.0
        total = e.sum(1, keepdims=True)
        soft = np.where(total > 0, e / np.where(total > 0, total, 1.0), 0.0)
        lse = np.where(total > 0, m + np.log(np.where(total > 0, total, 1.0)), 0.0)[:, 0]
        if score == "softmax":
            return soft, soft, np.ones_like(l), lse
        # sigmoids divided by the largest one's e^m where that is small, which leaves their shares alone
        s = np.where(m < 0, e / (1.0 + np.exp(l)), 1.0 / (1.0 + np.exp(-l)))
        s[~(l > -np.inf)] = 0.0
        total = s.sum(1, keepdims=True)
        p = np.where(total > 0, s / np.where(total > 0, total, 1.0), 0.0)
        return soft, p, 1.0 / (1.0 + np.exp(l)), lse


def _clean(logits):
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    return l


def losses(logits, idx, score="softmax", offsets=None):
    """(counts [S,E] int32, probs [S,E], balance [S], z [S])."""
    l = _clean(logits)
    T, E = l.shape
    k = idx.shape[1]
    offsets = [0, T] if offsets is None else list(offsets)
    S = len(offsets) - 1
    _, p, _, lse = _parts(l, score)
    counts, probs, balance, z = np.zeros((S, E), np.int32), np.zeros((S, E)), np.zeros(S), np.zeros(S)
    for s in range(S):
        a, b = offsets[s], offsets[s + 1]
        if a == b:
            continue
        chosen = idx[a:b].reshape(-1)
        counts[s] = np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
        probs[s] = p[a:b].mean(0)
        balance[s] = (counts[s] * (E / (k * (b - a))) * probs[s]).sum()
        z[s] = (lse[a:b] ** 2).mean()
    return counts, probs, balance, z


def weights(logits, idx, score="softmax", renormalize=True, scale=1.0):
    """The weights [T,k] of a given choice."""
    l = _clean(logits)
    soft, _, _, _ = _parts(l, score)
    s = soft if score == "softmax" else 1.0 / (1.0 + np.exp(-l))
    ok = (idx >= 0) & (idx < l.shape[1])
    w = np.where(ok, np.take_along_axis(s, np.where(ok, idx, 0), 1), 0.0)
    return scale * (w / w.sum(1, keepdims=True) if renormalize else w)


def backward(logits, idx, score="softmax", renormalize=True, scale=1.0, offsets=None, d_w=None, d_balance=None, d_z=None):
    """(d_logits [T,E], the sum of the magnitudes of the terms of each of its elements)."""
    l = _clean(logits)
    T, E = l.shape
    k = idx.shape[1]
    offsets = [0, T] if offsets is None else list(offsets)
    soft, p, slope, lse = _parts(l, score)
    counts = losses(logits, idx, score, offsets)[0]
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for s in range(len(offsets) - 1):
        a, b = offsets[s], offsets[s + 1]
        if a == b:
            continue
        if d_balance is not None:
            f = counts[s] * (E / (k * (b - a)))
            fp = (f * p[a:b]).sum(1, keepdims=True)
            c = d_balance[s] / (b - a) * p[a:b] * slope[a:b]
            d[a:b] += c * (f - fp)
            size[a:b] += np.abs(c) * (f + fp)
        if d_z is not None:
            c = d_z[s] / (b - a) * 2.0 * lse[a:b, None] * soft[a:b]
            d[a:b] += c
            size[a:b] += np.abs(c)
    if d_w is not None:
        for t in range(T):
            live = [j for j in range(k) if 0 <= idx[t, j] < E and l[t, idx[t, j]] > -np.inf]
            if not live:
                continue
            e = idx[t, live]
            g = np.asarray(d_w, np.float64)[t, live]
            if renormalize:
                m = l[t, e].max()
                if score == "softmax":
                    sc = np.where(l[t, e] == m, 1.0, np.exp(l[t, e] - m))
                else:
                    sc = np.where(m < 0, np.where(l[t, e] == m, 1.0, np.exp(l[t, e] - m)) / (1.0 + np.exp(l[t, e])),
                                  1.0 / (1.0 + np.exp(-l[t, e])))
                a = sc / sc.sum()
                h = slope[t, e] if score == "sigmoid" else 1.0
                dj, sj = scale * a * (g - (g * a).sum()) * h, np.abs(scale * a * h) * (np.abs(g) + np.abs(g * a).sum())
            else:
                sc = soft[t, e] if score == "softmax" else 1.0 / (1.0 + np.exp(-l[t, e]))
                dj = scale * g * sc * slope[t, e]
                sj = np.abs(dj)
                if score == "softmax":
                    d[t] -= soft[t] * dj.sum()
                    size[t] += soft[t] * sj.sum()
            np.add.at(d[t], e, dj)
            np.add.at(size[t], e, sj)
    return d, size
