"""Pins of the orthogonalised step's oracle: singular values one by one,
exact cases, the directions kept, planted mistakes."""

import numpy as np
import pytest

from oracle import muon as om


def _u(rows, cols, seed=0):
    return np.random.default_rng(seed).standard_normal((rows, cols))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (9, 1), (6, 6), (5, 40), (40, 5)])
@pytest.mark.parametrize("steps", [1, 3, 5])
def test_singular_values_follow_the_polynomial(rows, cols, steps):
    u = _u(rows, cols)
    U, s, V = np.linalg.svd(u, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    a, b, c = om.COEFFICIENTS
    want = s
    for _ in range(steps):
        want = a * want + b * want ** 3 + c * want ** 5
    np.testing.assert_allclose(om.orthogonalise(u, steps=steps), (U * want) @ V, rtol=0, atol=1e-11)
    np.testing.assert_allclose(om.growth(s * s, steps) * s, want, rtol=1e-12)


def test_five_steps_orthogonalise():
    s = np.linalg.svd(om.orthogonalise(_u(16, 400)), compute_uv=False)
    assert s.min() > 0.65 and s.max() < 1.25


def test_transpose_scale_and_zero():
    u = _u(4, 30)
    np.testing.assert_allclose(om.orthogonalise(u.T), om.orthogonalise(u).T, atol=1e-12)
    np.testing.assert_allclose(om.orthogonalise(u * 1e6, eps=1e-1), om.orthogonalise(u, eps=1e-7), atol=1e-6)
    assert (om.orthogonalise(np.zeros((3, 5))) == 0).all()


def test_step_by_hand():
    # 1 x 1: X = +-1, one step multiplies it by a + b + c
    a, b, c = om.COEFFICIENTS
    p, m, u = om.step(np.array([[2.0]]), np.array([[-3.0]]), np.array([[1.0]]), lr=0.1, momentum=0.5, weight_decay=0.2,
                      eps=1e-30, steps=1, grad_scale=2.0, lr_scale=3.0)
    assert m.item() == 0.5 - 6.0 and u.item() == -6.0 + 0.5 * -5.5
    assert p.item() == pytest.approx(2.0 * (1 - 0.02) + 0.1 * 3.0 * (a + b + c), rel=1e-14)
    p, m, u = om.step(np.array([[2.0]]), np.array([[4.0]]), np.array([[2.0]]), lr=0.1, nesterov=False)
    assert u.item() == m.item() == pytest.approx(5.9)


def test_planted_mistakes_are_seen():
    u, base = _u(8, 50), None
    base = om.orthogonalise(u)
    a, b, c = om.COEFFICIENTS
    for other in ((a, b, -c), (a, c, b), (a, b, 0.9 * c)):
        assert np.abs(om.orthogonalise(u, coefficients=other) - base).max() > 1e-3
    assert np.abs(om.orthogonalise(u, steps=4) - base).max() > 1e-3
