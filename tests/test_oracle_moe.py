"""Pins of the oracle of the token-chosen products: choices and weights by hand, experts and adapters in closed form."""
import numpy as np

from oracle import moe


def test_route_by_hand():
    ln = np.log
    a = np.array([[ln(1), ln(3), ln(4), ln(2)], [0.0, 1.0, 1.0, -np.inf], [-np.inf] * 4, [np.nan, 2.0, -np.inf, np.nan],
                  [np.inf, 0.0, np.inf, 1.0], [-0.0, 0.0, -1.0, -1.0]])
    ids, w = moe.route(a, 2, False)
    assert ids.tolist() == [[2, 1], [1, 2], [-1, -1], [1, -1], [0, 2], [0, 1]]
    e = np.e
    assert np.allclose(w, [[0.4, 0.3], [e / (1 + 2 * e)] * 2, [0, 0], [1, 0], [0.5, 0.5], [1 / (2 + 2 / e)] * 2])
    _, w = moe.route(a, 2, True)
    assert np.allclose(w, [[4 / 7, 3 / 7], [0.5, 0.5], [0, 0], [1, 0], [0.5, 0.5], [0.5, 0.5]])


def test_dense_by_hand():
    q = np.array([[8, 9, 0, 15]], np.uint8)
    assert moe.dense(q, np.array([[0.5, 2.0]]), np.array([[1.0, -1.0]])).tolist() == [[1.0, 1.5, -17.0, 13.0]]


def test_experts_closed_form():
    H, I = 4, 3
    r = np.random.default_rng(0)
    x = r.standard_normal((3, H))
    # expert 0: gate 0 -> silu 0; expert 1: gate rows of ones, up = the first input, down of ones
    gu = [np.concatenate([np.zeros((I, H)), r.standard_normal((I, H))]),
          np.concatenate([np.ones((I, H)), np.tile([1.0, 0, 0, 0], (I, 1))])]
    dn = [r.standard_normal((H, I)), np.ones((H, I))]
    ids = np.array([[0, -1], [1, 0], [1, 1]])
    w = np.array([[1.0, np.nan], [0.5, 2.0], [0.25, 0.5]])
    y = moe.experts(x, ids, w, gu, dn)
    s = x.sum(1)
    one = I * s / (1 + np.exp(-s)) * x[:, 0]
    assert np.allclose(y, np.stack([np.zeros(H), np.full(H, 0.5 * one[1]), np.full(H, 0.75 * one[2])]))


def test_adapters_are_dense_matrices():
    r = np.random.default_rng(1)
    x, base = r.standard_normal((5, 6)), r.standard_normal((5, 4))
    a, b = r.standard_normal((2, 3, 6)), r.standard_normal((2, 4, 3))
    y = moe.adapters(x, base, np.array([0, 1, -1, 1, 0]), a, b, np.array([3, 1]), np.array([2.0, -1.0]))
    W = [2.0 * b[0] @ a[0], -np.outer(b[1][:, 0], a[1][0])]
    assert np.allclose(y, base + np.stack([W[0] @ x[0], W[1] @ x[1], 0 * base[2], W[1] @ x[3], W[0] @ x[4]]))
