"""Pins of the routing and AdamW oracles (oracle/routing.py, oracle/adamw.py)
that need no GPU: hand cases, finite differences, an independent
implementation, and planted mistakes that the pins must notice."""

import numpy as np
import pytest
import torch

from oracle import adamw as oa
from oracle import routing as orr

NAN, INF = float("nan"), float("inf")


def test_route_hand_cases():
    x = np.array([[0.0, 2.0, 2.0, 1.0], [-INF, 3.0, -INF, -INF], [-INF] * 4, [1.0, 1.0, 1.0, 1.0]])
    ids, w = orr.route(x, 2, renorm=False)
    assert ids.tolist() == [[1, 2], [1, -1], [-1, -1], [0, 1]]
    z = 1 + 2 * np.e ** 2 + np.e
    assert np.allclose(w, [[np.e ** 2 / z] * 2, [1, 0], [0, 0], [0.25, 0.25]], rtol=1e-15)
    ids, w = orr.route(x, 3, renorm=True)
    z = 2 * np.e ** 2 + np.e
    assert ids[0].tolist() == [1, 2, 3] and np.allclose(w[0], [np.e ** 2 / z, np.e ** 2 / z, np.e / z])
    assert np.allclose(w.sum(1), [1, 1, 0, 1])


def _fd_route(x, ids, dw, renorm, h=1e-6):
    """Central differences of sum(dw * weights) with the choice held fixed."""
    def loss(y):
        total = 0.0
        for t in range(y.shape[0]):
            p = np.exp(y[t] - y[t].max())
            c = [e for e in ids[t] if e >= 0]
            z = p[c].sum() if renorm else p.sum()
            total += sum(d * p[e] / z for e, d in zip(ids[t], dw[t]) if e >= 0)
        return total
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = (loss(a) - loss(b)) / (2 * h)
    return out


@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(renorm):
    rng = np.random.default_rng(1)
    x, dw = rng.standard_normal((4, 7)), rng.standard_normal((4, 3))
    ids, _ = orr.route(x, 3, renorm)
    ids[2, 2] = -1
    got, fd = orr.route_backward(x, ids, dw, renorm), _fd_route(x, ids, dw, renorm)
    # differences with step h: h^2 / 6 of a third derivative below 10, and
    # rounding of 2^-52 * 10 / h
    assert np.abs(got - fd).max() < 1e-8
    # a gradient without the softmax's second term must not pass
    p = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    up = np.zeros_like(x)
    for t in range(4):
        up[t, [e for e in ids[t] if e >= 0]] = [d for e, d in zip(ids[t], dw[t]) if e >= 0]
    assert np.abs(p * up - fd).max() > 1e-3


def test_dispatch_is_the_stable_argsort():
    rng = np.random.default_rng(2)
    ids = rng.integers(-1, 6, (37, 3))          # -1 and 5 are outside E = 5
    off, rows, slots = orr.dispatch(ids, 5)
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < 5), flat, 5)
    order = np.argsort(key, kind="stable")[: off[-1]]
    assert np.array_equal(slots, order)
    assert np.array_equal(off, np.searchsorted(np.sort(key), np.arange(6)))
    assert np.array_equal(rows.reshape(-1)[slots], np.arange(off[-1])) and (rows.reshape(-1)[key == 5] == -1).all()
    assert not np.array_equal(slots, np.argsort(-key, kind="stable")[: off[-1]])


def test_combine_and_its_gradient():
    rng = np.random.default_rng(3)
    T, k, D, E = 9, 2, 5, 4
    ids = rng.integers(-1, E, (T, k))
    off, rows, slots = orr.dispatch(ids, E)
    Ys, w, dY = rng.standard_normal((T * k, D)), rng.standard_normal((T, k)), rng.standard_normal((T, D))
    Ys[off[-1]:], w[rows < 0] = NAN, NAN          # never read
    base = rng.standard_normal((T, D))
    Y = orr.combine(Ys, rows, w, base)
    M = np.zeros((T, T * k))                      # the same as a matrix product
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                M[t, rows[t, j]] += w[t, j]
    live = np.arange(T * k) < off[-1]
    assert np.allclose(Y, base + M[:, live] @ Ys[live])
    dYs, dw = orr.combine_backward(dY, Ys, rows, w)
    assert np.allclose(dYs[live], M[:, live].T @ dY) and np.isnan(dYs[~live]).all()
    h = 1e-6
    for t, j in ((0, 0), (4, 1), (8, 0)):
        if rows[t, j] < 0:
            assert dw[t, j] == 0
            continue
        a, b = w.copy(), w.copy()
        a[t, j] += h
        b[t, j] -= h
        fd = ((orr.combine(Ys, rows, a) - orr.combine(Ys, rows, b)) * dY).sum() / (2 * h)
        assert abs(fd - dw[t, j]) < 1e-8
    with pytest.raises(AssertionError):           # swapped choices do not pass
        assert np.allclose(orr.combine(Ys, rows[:, ::-1], w, base), Y)


def test_adamw_step_against_torch():
    rng = np.random.default_rng(4)
    p = torch.tensor(rng.standard_normal(50), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.tensor(g)
        opt.step()
        q, m, v = oa.step(q, g / 4, m, v, t, 3e-3, 0.8, 0.95, 1e-6, 0.1, grad_scale=4.0)
        assert np.allclose(q, p.detach().numpy(), rtol=1e-12, atol=0)
    # the first step from zero states moves each element by lr against its sign
    q, _, _ = oa.step(np.zeros(3), [2.0, -1e-3, 0.0], np.zeros(3), np.zeros(3), 1, 0.5, eps=0.0 + 1e-30)
    assert np.allclose(q, [-0.5, 0.5, 0.0])


def test_e4m3_codes():
    table = oa.code_values()
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(codes.double().numpy(), table, equal_nan=True)
    # exact round trip of every value under a scale that is a power of two
    vals = np.concatenate([table[:127], -table[1:127]]) * 2.0 ** -20
    c, s = oa.encode(vals)
    assert s[0] == 2.0 ** -20 and np.array_equal(oa.decode(c, s), vals)
    # nearest code: half a step, and torch's conversion of the same quotients
    x = np.random.default_rng(5).standard_normal(700) * np.exp(np.random.default_rng(6).standard_normal(700) * 4)
    c, s = oa.encode(x)
    scale = np.repeat(s, 256)[:700]
    assert (np.abs(oa.decode(c, s) - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 1e-12)).all()
    t = torch.tensor(x / scale).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # (torch rounds the quotient to float first, so a tie may go the other way)
    assert (np.abs(t.astype(int) - c.astype(int)) <= 1).all() and (t == c).mean() > 0.99
    # roots above zero keep a code; truncation instead of rounding is noticed
    c, s = oa.encode([1.0, 1e-9, 0.0], root=True)
    assert c[1] == 1 and c[2] == 0 and oa.encode([1.0, 1e-9])[0][1] == 0
    down = np.abs(x) / scale
    down = np.array([table[:127][table[:127] <= q][-1] for q in down]) * scale
    assert (np.abs(down - np.abs(x)) > np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 1e-12)).any()
    assert oa.encode(np.full(3, 1e-31))[1][0] == 0.0


def test_route_backward_of_rows_without_ids():
    """Zeros, whatever the logits are."""
    x = np.array([[NAN, 1.0, 2.0], [np.inf, 0.0, -1.0], [0.5, 1.0, 2.0]])
    ids = np.array([[-1, 3], [7, -5], [2, -1]])
    for renorm in (False, True):
        d = orr.route_backward(x, ids, np.ones((3, 2)), renorm)
        assert (d[:2] == 0).all() and np.isfinite(d).all()
    assert (orr.route_backward(x, ids, np.ones((3, 2)), False)[2] != 0).all()


def test_e4m3_codes_by_chance():
    """encode_random: codes themselves stay, the values around a number come
    in the shares that keep its mean (its square's, for roots)."""
    rng = np.random.default_rng(7)
    table = oa.code_values()
    exact = np.concatenate([table[:127], -table[1:127]]) * 2.0 ** -20
    for u in (0.0, 0.5, 1 - 2.0 ** -53):
        c, s = oa.encode_random(exact, np.full(exact.size, u))
        assert np.array_equal(oa.decode(c, s), exact)
    n, steps = 256, 4096
    x = np.abs(rng.standard_normal(n)) * np.exp(rng.standard_normal(n) * 3)
    u = (np.arange(steps) + 0.5) / steps                  # every share, to half a grid step
    for root in (False, True):
        power = 2 if root else 1
        c, s = zip(*(oa.encode_random(x, np.full(n, q), root) for q in u))
        vals = np.stack([oa.decode(a, b) for a, b in zip(c, s)])
        gap = vals.max(0) ** power - vals.min(0) ** power
        want = np.maximum(x, s[0][0] * 2.0 ** -9) ** power if root else x
        assert (np.abs((vals ** power).mean(0) - want) <= gap * 0.51 / steps + 1e-12 * want).all()
        step = np.maximum(want ** (1 / power) / 8, s[0][0] * 2.0 ** -9)     # codes beside x: at most this apart,
        apart = step * (2 * want ** 0.5 + step) if root else step         # their squares (x + step)^2 - x^2
        assert (gap <= apart * (1 + 1e-9)).all()
    with pytest.raises(AssertionError):                   # the chance of the values is not that of the squares
        c, s = zip(*(oa.encode_random(x, np.full(n, q), False) for q in u))
        vals = np.stack([oa.decode(a, b) for a, b in zip(c, s)])
        assert (np.abs((vals ** 2).mean(0) - x ** 2) <= gap * 0.51 / steps + 1e-12).all()


def test_stored_root_follows_only_by_chance():
    """v = b2 v + (1 - b2) g^2 with its root stored as codes at every step,
    gradients of half the elements 20 times smaller after a third: by chance
    the mean of v is the formula's; at the nearest code it stays."""
    rng = np.random.default_rng(8)
    n, b2, ends = 256 * 16, 0.99, {}
    for how in ("chance", "near"):
        v, want = np.zeros(n), np.zeros(n)
        for t in range(900):
            g2 = np.where((np.arange(n) % 2 == 0) & (t >= 300), 0.05, 1.0) ** 2
            v, want = b2 * v + (1 - b2) * g2, b2 * want + (1 - b2) * g2
            c, s = oa.encode_random(np.sqrt(v), rng.random(n) if how == "chance" else np.full(n, 0.5), True)
            v = oa.decode(c, s) ** 2
        ends[how] = v[::2].mean() / want[::2].mean()
    # (an element's v has a standard deviation of the size of its mean at most here: 2048 of them, 6 of the mean's)
    assert abs(ends["chance"] - 1) < 6 / 2048 ** 0.5 and ends["near"] > 50, ends
