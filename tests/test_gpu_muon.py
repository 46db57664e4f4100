"""The orthogonalised step on the GPU against the float64 oracle
(oracle/muon.py).

Tolerances, derived: u = 2^-24 is fp32's half step, h = 2^-8 bf16's.  Of X,
with X_0 the normalised update (its norm is 1), sigma its singular values, q
the growth of a direction (X = Q X_0), KB <= 256 columns to a float sum:
 - the update itself: three roundings, 3 u of it; so Q's argument A = X_0
   X_0^T is off by 6 u, and by the float sums, whose roundings add up like a
   random walk: 4 u sqrt(KB) of |X_0| |X_0|^T.  To first order an error E of A
   changes X by sigma_j (q_i - q_j) / (s_i - s_j) E_ij in the singular
   directions (s = sigma^2; q' where i = j): at most K |E| with K the largest
   of these factors;
 - Q is stored as float after each step: u |Q| each, |X_0| = 1;
 - Q X_0 in float: 4 u sqrt(S) of |Q| |X_0|, and 3 u of X_0 times the largest
   growth.
All norms are Frobenius norms, and no element is off by more than the norm.
m: 3 u of the magnitudes.  p: that of X times the rate, 4 u of the terms, h of
the result for bf16."""

import numpy as np
import pytest

from oracle import muon as om
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8


def _srl():
    import sparse_rank_linear_amd as srl

    return srl


def _f64(t):
    return t.detach().double().cpu().numpy()


def x_tolerance(u, steps=5, eps=1e-7):
    """How far X may be off, in norm."""
    X = u if u.shape[0] <= u.shape[1] else u.T
    norm = np.sqrt((X * X).sum())
    if norm == 0:
        return 0.0
    X = X / (norm + eps)
    s, V = np.linalg.eigh(X @ X.T)
    s = np.maximum(s, 0.0)
    q = om.growth(s, steps)
    d = 1e-6 * max(s.max(), 1e-30)
    slope = (om.growth(s + d, steps) - om.growth(np.maximum(s - d, 0), steps)) / (s + d - np.maximum(s - d, 0))
    gap = s[:, None] - s[None, :]
    near = np.abs(gap) < 1e-9 * s.max() + 1e-300
    factor = np.where(near, (slope[:, None] + slope[None, :]) / 2, (q[:, None] - q[None, :]) / np.where(near, 1.0, gap))
    K = np.abs(factor * np.sqrt(s)[None, :]).max()
    Q = (V * q) @ V.T
    sums = 4 * U * 16 * np.linalg.norm(np.abs(X) @ np.abs(X).T)
    return (K * (sums + 6 * U) + steps * U * np.linalg.norm(Q) + 3 * U * np.abs(q).max()
            + 4 * U * 16 * np.linalg.norm(np.abs(Q) @ np.abs(X)) + 1e-30)


def _gradient(rows, cols, kind, rng):
    if kind == "noise":
        return rng.standard_normal((rows, cols))
    if kind == "signal":         # a few strong directions and noise
        few = min(4, rows, cols)
        return rng.standard_normal((rows, few)) @ rng.standard_normal((few, cols)) + 0.05 * rng.standard_normal(
            (rows, cols))
    if kind == "low":            # of low rank, with rows and columns of zeros
        few = max(1, min(rows, cols) // 3)
        x = rng.standard_normal((rows, few)) @ rng.standard_normal((few, cols))
        x[rows // 2] = 0
        x[:, cols // 3] = 0
        return x
    return np.zeros((rows, cols))


class Group:
    def __init__(self, shapes, p_half=False, g_half=False, master=False, kind="noise", seed=0, fresh=False):
        import torch

        srl, rng = _srl(), np.random.default_rng(seed)
        pt, gt = torch.bfloat16 if p_half else torch.float32, torch.bfloat16 if g_half else torch.float32
        up = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).cuda().to(t)
        self.params = [up(rng.standard_normal(s) * 0.02, pt) for s in shapes]
        kinds = kind if isinstance(kind, list) else [kind] * len(shapes)
        self.grads = [up(_gradient(*s, k, rng) * 10.0 ** (-4 + i % 5), gt) for i, (s, k) in enumerate(zip(shapes, kinds))]
        self.st = srl.muon_states(self.params, master=master)
        if not fresh:
            for i, (m, s, k) in enumerate(zip(self.st["m"], shapes, kinds)):
                m.copy_(up(_gradient(*s, k, rng) * 10.0 ** (-4 + i % 5) * 3, torch.float32))
        if master:
            for w in self.st["master"]:
                w.add_(1e-5)
        self.master, self.p_half = master, p_half
        self.lr_scale = [1.0 + 0.5 * (i % 3) for i in range(len(shapes))]
        self.plan = srl.muon_plan(self.params, self.grads, lr_scale=self.lr_scale, **self.st)
        self.keep()

    def keep(self):
        src = self.st["master"] if self.master else self.params
        self.before = [(_f64(p), _f64(g), _f64(m)) for p, g, m in zip(src, self.grads, self.st["m"])]

    def check(self, lr, weight_decay=0.0, momentum=0.95, nesterov=True, steps=5, grad_scale=1.0):
        for i, (p0, g, m0) in enumerate(self.before):
            p, m, u = om.step(p0, g, m0, lr, momentum, nesterov, weight_decay, 1e-7, steps, grad_scale=grad_scale,
                              lr_scale=self.lr_scale[i])
            tm = 3 * U * (np.abs(momentum * m0) + np.abs(g * grad_scale)) + 1e-40
            assert (np.abs(_f64(self.st["m"][i]) - m) <= tm).all(), (i, p0.shape)
            tx = x_tolerance(u, steps)
            rate = lr * self.lr_scale[i]
            X = (p0 * (1 - lr * weight_decay) - p) / rate if rate else np.zeros_like(p)
            tol = 4 * U * (np.abs(p0) + rate * np.abs(X))
            got = _f64(self.st["master"][i] if self.master else self.params[i])
            off = np.abs(got - p)
            half = self.p_half and not self.master
            bound = rate * tx + tol + (H * np.abs(p) * (1 + H) + H * rate * tx if half else 0)
            say(f"  {p0.shape}: X off by {np.linalg.norm(got - p) / max(rate, 1e-30):.2e} of {np.linalg.norm(X):.2e}, "
                f"allowed {tx:.2e}")
            assert (off <= bound).all(), (i, p0.shape, off.max())
            if not half:
                assert np.linalg.norm(got - p) <= rate * tx + np.linalg.norm(tol)
            if self.master:
                assert (_f64(self.params[i]) == _f64(self.st["master"][i].to(self.params[i].dtype))).all()


# every class of short side and both orientations: the sizes around its
# borders, rows that start anywhere, several pieces of the long side
SHAPES = [(1, 1), (1, 7), (7, 1), (3, 3), (16, 16), (5, 300), (300, 5), (16, 1000), (1001, 15), (17, 515), (515, 32),
          (33, 130), (130, 48), (49, 777), (777, 64), (65, 901), (901, 80), (80, 1024), (81, 400), (400, 96), (97, 333),
          (333, 112), (113, 500), (500, 128), (129, 450), (450, 160), (161, 400), (400, 192), (193, 300), (301, 253),
          (256, 512), (256, 256)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_x_alone(rows, cols):
    """p = -X from zero parameters."""
    import torch

    grp = Group([(rows, cols)], seed=rows + cols)
    grp.params[0].zero_()
    grp.keep()
    _srl().muon_step(grp.plan, 1.0)
    torch.cuda.synchronize()
    grp.check(1.0)


@pytest.mark.parametrize("kind", ["signal", "low", "zero"])
@pytest.mark.parametrize("rows,cols", [(16, 640), (1111, 80), (112, 999), (700, 130), (256, 1025)])
def test_spectra(rows, cols, kind):
    grp = Group([(rows, cols)], kind=kind, seed=rows)
    grp.params[0].zero_()
    grp.keep()
    _srl().muon_step(grp.plan, 1.0)
    grp.check(1.0)


TYPES = [(False, False, False), (False, True, False), (True, False, False), (True, True, False), (True, False, True),
         (True, True, True)]


@pytest.mark.parametrize("p_half,g_half,master", TYPES)
def test_types_and_mixed_shapes(p_half, g_half, master):
    """Matrices of several classes, an empty one among them, in one plan; two
    steps, the second from what the first left."""
    shapes = [(80, 2048), (0, 5), (1408, 80), (16, 4096), (4097, 16), (7, 9), (200, 640), (641, 129), (3, 0), (33, 64)]
    grp = Group(shapes, p_half, g_half, master, kind=["noise", "signal"] * 5, seed=3)
    for k in range(2):
        grp.keep()
        _srl().muon_step(grp.plan, 0.01, weight_decay=0.1, grad_scale=0.5)
        grp.check(0.01, 0.1, grad_scale=0.5)


@pytest.mark.parametrize("steps,nesterov,momentum", [(1, True, 0.9), (2, False, 0.0), (3, True, 0.0), (4, False, 0.99),
                                                     (6, True, 0.95)])
def test_arguments(steps, nesterov, momentum):
    grp = Group([(20, 300), (300, 150), (16, 16)], seed=steps)
    _srl().muon_step(grp.plan, 0.3, steps=steps, nesterov=nesterov, momentum=momentum)
    grp.check(0.3, steps=steps, nesterov=nesterov, momentum=momentum)
