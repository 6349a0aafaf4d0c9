"""Pins of the gate and norm oracle: closed forms, brute force and limits."""
import itertools

import numpy as np
import pytest

from oracle import layer as ol
from oracle import moe as omoe


def test_plain_softmax_gate_is_the_blocks_gate():
    rng = np.random.default_rng(1)
    l = rng.normal(size=(40, 24)).astype(np.float32)
    idx, w = ol.gate(l, 5)
    np.testing.assert_array_equal(idx, omoe.topk_select(l, 5))
    np.testing.assert_allclose(w, omoe.gate_weights(l, idx), rtol=1e-14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_gate_against_brute_force_over_group_subsets(score, group_top):
    """The kept groups are the subset of that many groups with the largest total value, the chosen experts
    the subset of theirs with the largest total choice."""
    rng = np.random.default_rng(2)
    G, gs, kept, k = 4, 3, 2, 3
    l = rng.normal(size=(30, G * gs)).astype(np.float32)
    b = rng.normal(size=G * gs).astype(np.float32) * 0.3
    idx, w = ol.gate(l, k, score, b, G, kept, group_top, renormalize=False, scale=3.0)
    for t in range(len(l)):
        x = l[t].astype(np.float64)
        s = 1 / (1 + np.exp(-x)) if score == "sigmoid" else np.exp(x) / np.exp(x).sum()
        c = s + b
        val = [np.sort(c[g * gs:(g + 1) * gs])[::-1][:group_top].sum() for g in range(G)]
        best = max(itertools.combinations(range(G), kept), key=lambda S: sum(val[g] for g in S))
        cand = [e for g in best for e in range(g * gs, (g + 1) * gs)]
        pick = max(itertools.combinations(cand, k), key=lambda S: sum(c[e] for e in S))
        assert set(idx[t]) == set(pick)
        assert list(idx[t]) == sorted(pick, key=lambda e: -c[e])
        np.testing.assert_allclose(w[t], 3.0 * s[idx[t]], rtol=1e-13)


def test_gate_limits():
    inf = np.inf
    idx, w = ol.gate(np.array([[-inf, np.nan, -inf, 2.0]], np.float32), 2, "sigmoid")
    assert idx.tolist() == [[3, -1]] and w.tolist() == [[1.0, 0.0]]
    idx, w = ol.gate(np.full((1, 3), -inf, np.float32), 2)
    assert idx.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]
    idx, w = ol.gate(np.array([[inf, 1.0, inf]], np.float32), 3, renormalize=False)
    assert idx.tolist() == [[0, 2, 1]] and w.tolist() == [[0.5, 0.5, 0.0]]
    # sigmoids that underflow keep their ratio when renormalised
    idx, w = ol.gate(np.array([[-2000.0, -2001.0]], np.float32), 2, "sigmoid")
    np.testing.assert_allclose(w[0], [1 / (1 + np.exp(-1)), np.exp(-1) / (1 + np.exp(-1))], rtol=1e-14)
    # an expert out of service still counts in the softmax
    idx, w = ol.gate(np.zeros((1, 4), np.float32), 2, balance=[0, -inf, 0, 0], renormalize=False)
    assert idx.tolist() == [[0, 2]] and w.tolist() == [[0.25, 0.25]]


def test_rmsnorm_and_combine_closed_forms():
    np.testing.assert_allclose(ol.rmsnorm([[3.0, 4.0]], [1.0, 2.0], 0.0), [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    y = np.arange(8.0).reshape(4, 2)
    z, mag = ol.combine(y, np.array([[1, -1]]), np.array([[-2.0, 5.0]]), 1)
    assert z.tolist() == [[-2 * 2 + 4, -2 * 3 + 5]] and mag.tolist() == [[4 + 4, 6 + 5]]
