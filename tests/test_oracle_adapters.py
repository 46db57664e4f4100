"""Pins of the adapters' oracle: hand cases, the layer that a user would
build from one adapter (oracle/salr.py's forward and oracle/backward.py's
gradients with nothing kept), central differences, planted mistakes."""

import numpy as np
import pytest

from oracle import adapters as oa


def _case(M=7, count=3, r=4, K=8, N=5, seed=0):
    g = np.random.default_rng(seed)
    a, b = g.standard_normal((count, r, K)), g.standard_normal((count, N, r))
    ids = np.array([0, 2, -1, 2, 0, count, 2][:M])
    return a, b, ids, np.array([4, 3, 2][:count]), np.array([1.0, 0.5, -2.0][:count]), g.standard_normal((M, K)), \
        g.standard_normal((M, N)), g.standard_normal((M, K)), g.standard_normal((M, N))


def test_hand_case():
    a = np.array([[[1.0, 2.0]], [[10.0, 0.0]]])           # two adapters, rank 1, K = 2
    b = np.array([[[3.0]], [[1.0]]])                      # N = 1
    X, base = np.array([[1.0, 1.0], [2.0, 5.0], [7.0, 7.0]]), np.array([[0.5], [0.0], [9.0]])
    Y = oa.forward(a, b, [0, 1, 2], [1, 1], [1.0, 0.1], X, base)
    assert Y.ravel().tolist() == [0.5 + 9.0, 0.1 * 20.0, 9.0]
    dX, dA, dB = oa.backward(a, b, [0, 1, 2], [1, 1], [1.0, 0.1], X, np.ones((3, 1)), np.zeros((3, 2)))
    assert dX.tolist() == [[3.0, 6.0], [1.0, 0.0], [0.0, 0.0]]
    assert dA.ravel().tolist() == [3.0, 3.0, pytest.approx(0.2), pytest.approx(0.5)]
    assert dB.ravel().tolist() == [3.0, 2.0]


def test_matrix_form():
    a, b, ids, ranks, scales, X, dY, bx, by = _case()
    Y = oa.forward(a, b, ids, ranks, scales, X, by)
    dX, dA, dB = oa.backward(a, b, ids, ranks, scales, X, dY, bx)
    for q in range(3):
        at, n = np.flatnonzero(ids == q), ranks[q]
        A, B = a[q, :n].T, b[q, :, :n].T * scales[q]      # X A B
        np.testing.assert_allclose(Y[at], by[at] + X[at] @ A @ B, rtol=1e-12)
        np.testing.assert_allclose(dX[at], bx[at] + dY[at] @ B.T @ A.T, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(dA[q, :n], (X[at].T @ dY[at] @ B.T).T, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(dB[q, :, :n], scales[q] * ((X[at] @ A).T @ dY[at]).T, rtol=1e-12, atol=1e-12)
        assert (dA[q, n:] == 0).all() and (dB[q, :, n:] == 0).all()
    np.testing.assert_array_equal(Y[[2, 5]], by[[2, 5]])
    assert (dA[1] == 0).all() and (dB[1] == 0).all()      # no token names it


@pytest.mark.parametrize("which", ["a", "b", "X"])
def test_differences(which):
    a, b, ids, ranks, scales, X, dY, bx, by = _case()
    dX, dA, dB = oa.backward(a, b, ids, ranks, scales, X, dY, np.zeros_like(X))
    at, grad = {"a": (a, dA), "b": (b, dB), "X": (X, dX)}[which]
    loss = lambda: float((dY * oa.forward(a, b, ids, ranks, scales, X, by)).sum())
    for i in np.ndindex(at.shape):                        # (linear in each: differences are exact)
        keep = at[i]
        at[i] = keep + 0.5
        up = loss()
        at[i] = keep - 0.5
        assert up - loss() == pytest.approx(grad[i], rel=1e-10, abs=1e-10)
        at[i] = keep


def test_planted_mistakes_are_seen():
    a, b, ids, ranks, scales, X, dY, bx, by = _case()
    Y = oa.forward(a, b, ids, ranks, scales, X, by)
    assert np.abs(oa.forward(a, b, ids, ranks, np.ones(3), X, by) - Y).max() > 0.1
    assert np.abs(oa.forward(a, b, ids, [4, 4, 4], scales, X, by) - Y).max() > 0.1
    assert np.abs(oa.forward(a, b, np.roll(ids, 1), ranks, scales, X, by) - Y).max() > 0.1


def test_plan():
    off, order = oa.plan([2, -1, 0, 2, 7, 0], 3)
    assert off.tolist() == [0, 2, 2, 4, 6] and order.tolist() == [2, 5, 0, 3, 1, 4]
