"""The oracles of the branch, the balance loss, the gate's gradient and int8 rows, by hand and by differences."""
import numpy as np
import pytest

from oracle import balance as ob
from oracle import int8 as o8
from oracle import layer as ol


def test_branch_by_hand():
    u, res = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    # rms of (3, 4) is sqrt(12.5)
    z = ol.branch(u, res, norm=[2.0, 1.0], eps=0.0, gate=[1.0, 0.5], token_gate=[2.0], scale=0.25, residual_scale=3.0)
    r = np.sqrt(12.5)
    np.testing.assert_allclose(z, [[3.0 + 0.5 * 6.0 / r, -3.0 + 0.25 * 4.0 / r]])
    np.testing.assert_array_equal(ol.branch(u, res), u + res)
    np.testing.assert_array_equal(ol.branch(u), u)


def test_balance_of_an_even_and_of_a_one_sided_load():
    E, k = 4, 2
    l = np.zeros((6, E))
    even = np.array([[0, 1], [2, 3]] * 3)
    counts, probs, balance, z = ob.losses(l, even)
    assert (counts == 3).all() and np.allclose(probs, 0.25) and np.allclose(balance, 1.0) and np.allclose(z, np.log(4) ** 2)
    one = np.zeros((6, 2), np.int64)
    one[:, 1] = -1
    counts, _, balance, _ = ob.losses(l, one)
    assert counts.tolist() == [[6, 0, 0, 0]] and np.allclose(balance, 6 * E / (k * 6) * 0.25)
    # two sequences, an empty one between them, and tokens outside
    counts, probs, balance, z = ob.losses(l, even, offsets=[1, 3, 3, 5])
    assert counts.sum(1).tolist() == [4, 0, 4] and balance[1] == 0 and z[1] == 0 and (probs[1] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("shift", [0.0, -80.0])
def test_gradient_against_differences(score, renormalize, shift):
    rng = np.random.default_rng(3)
    T, E, k = 7, 5, 2
    l = rng.normal(size=(T, E)) * 1.5 + (shift if renormalize else 0.0)
    idx = np.argsort(-l, 1)[:, :k].copy()
    idx[1, 1] = -1
    idx[2, 1] = idx[2, 0]                    # the same expert twice
    l[3, 4] = -np.inf
    off = [1, 4, 4, 6]
    dw, db, dz = rng.normal(size=(T, k)), rng.normal(size=3), rng.normal(size=3) * 0.1

    def total(l):
        _, _, b, z = ob.losses(l, idx, score, off)
        return (ob.weights(l, idx, score, renormalize, 1.5) * dw).sum() + (b * db).sum() + (z * dz).sum()

    d, size = ob.backward(l, idx, score, renormalize, 1.5, off, dw, db, dz)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert d[t, e] == 0
                continue
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            # error of a central difference: h^2 / 6 third derivatives, and the losses' rounding over h
            assert abs((total(up) - total(down)) / (2 * h) - d[t, e]) < 1e-8 + 1e-6 * size[t, e] + 1e-16 * abs(total(l)) / h * 10


def test_int8_rows_by_hand():
    x = np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1e-44, 0, 0, 0], [np.inf, 1, 2, 3], [np.nan, 1, 2, 3]], np.float32)
    q, s = o8.rows(x)
    assert q[0].tolist() == [127, -64, 0, 2] and s[0] == 1        # ties go to the even code
    assert q[1].tolist() == [0] * 4 and s[1] == 1
    assert q[2].tolist() == [0] * 4 and s[2] == np.float32(2.0 ** -126)
    assert (q[3:] == 0).all() and np.isnan(s[3:]).all()
    w = np.array([[1, 2, 3, 4], [-1, 0, 0, 0]], np.int8)
    np.testing.assert_array_equal(o8.product(q[:1], s[:1], w, np.array([0.5, 2.0], np.float32)),
                                  [[(127 - 128 + 0 + 8) * 0.5, -254.0]])
