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


def test_training_steps_tell_mistakes_apart():
    """The training of tests/test_gpu_muon.py's
    test_training_steps_follow_the_definition with mistakes planted in a step:
    a wrong direction or rate is ten times what that test allows at every step;
    a momentum that is not carried or not looked ahead with is seen at most
    steps by the parameters, and the first at every step by the momentum."""
    from tests.test_gpu_muon import U, x_tolerance

    rng = np.random.default_rng(0)
    W = rng.standard_normal((96, 16)) @ rng.standard_normal((16, 64))
    P = [rng.standard_normal((96, 16)) * 0.1, rng.standard_normal((16, 64)) * 0.1]
    M, lr, scales, seen = [np.zeros_like(p) for p in P], 0.05, (1.0, 1.5), {}
    for k in range(20):
        R = P[0] @ P[1] - W
        G = [R @ P[1].T, P[0].T @ R]
        for i in (0, 1):
            go = lambda g, m, **kw: om.step(P[i], g, m, lr, lr_scale=scales[i], **kw)
            p, m, u = go(G[i], M[i])
            bound = lr * scales[i] * x_tolerance(u) + 4 * U * np.linalg.norm(np.abs(P[i]) + np.abs(p - P[i]))
            wrong = {"the other direction": go(-G[i], -M[i]), "the gradient's sign": go(-G[i], M[i]),
                     "half the rate": om.step(P[i], G[i], M[i], lr / 2, lr_scale=scales[i])}
            for name, (q, _, _) in wrong.items():
                if k == 0 or name != "the gradient's sign":      # (later the momentum outweighs it)
                    assert np.linalg.norm(q - p) > 10 * bound, (k, i, name)
                seen.setdefault(name, []).append(np.linalg.norm(q - p) > bound)
            if k > 0:
                lost = go(G[i], 0 * M[i])
                assert (np.abs(lost[1] - m) > 10 * 3 * U * (np.abs(0.95 * M[i]) + np.abs(G[i]))).any()
                for name, q in (("no momentum", lost[0]), ("no Nesterov", go(G[i], M[i], nesterov=False)[0])):
                    seen.setdefault(name, []).append(np.linalg.norm(q - p) > bound)
            P[i], M[i] = p, m
    assert all(np.mean(v) > 0.8 for v in seen.values()), {n: np.mean(v) for n, v in seen.items()}
