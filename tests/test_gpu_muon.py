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
        self.grads = [up(_gradient(*s, k, rng) * 10.0 ** (-4 + i % 5), gt)
                      for i, (s, k) in enumerate(zip(shapes, kinds))]
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


def test_as_exact_as_float_steps():
    """Not much further from the definition than Newton-Schulz steps on X
    itself in float, also where singular values differ a hundredfold: ten
    times their error and 2^-20 (the sums over A's small eigenvalues)."""
    import torch

    for kind in ("noise", "signal"):
        grp = Group([(80, 2048), (1408, 80), (250, 900)], kind=kind, seed=11)
        for p in grp.params:
            p.zero_()
        grp.keep()
        _srl().muon_step(grp.plan, 1.0)
        for i, (p0, g, m0) in enumerate(grp.before):
            want = om.step(p0, g, m0, 1.0, lr_scale=grp.lr_scale[i])[0]
            u = torch.from_numpy(g + 0.95 * (0.95 * m0 + g)).float().cuda()
            x = u / (u.norm() + 1e-7)
            x = x if x.shape[0] <= x.shape[1] else x.t().contiguous()
            for _ in range(5):
                A = x @ x.t()
                x = om.COEFFICIENTS[0] * x + (om.COEFFICIENTS[1] * A + om.COEFFICIENTS[2] * (A @ A)) @ x
            x = x if x.shape == u.shape else x.t()
            norm = np.linalg.norm(want)
            plain = np.linalg.norm(_f64(x) * -grp.lr_scale[i] - want) / norm
            mine = np.linalg.norm(_f64(grp.params[i]) - want) / norm
            say(f"  {kind} {p0.shape}: float steps {plain:.1e}, here {mine:.1e}")
            assert mine <= 10 * plain + 2.0 ** -20


def test_training_shrinks_a_residual():
    """The step as an optimizer's: gradients of |A - W|^2 for a factored A."""
    import torch

    srl = _srl()
    torch.manual_seed(0)
    W = torch.randn(96, 16, device="cuda") @ torch.randn(16, 64, device="cuda")
    P = [torch.randn(96, 16, device="cuda") * 0.1, torch.randn(16, 64, device="cuda") * 0.1]
    G = [torch.empty_like(p) for p in P]
    plan = srl.muon_plan(P, G, **srl.muon_states(P))
    for _ in range(20):
        R = P[0] @ P[1] - W
        G[0].copy_(R @ P[1].t())
        G[1].copy_(P[0].t() @ R)
        srl.muon_step(plan, 0.05)
        assert all(torch.isfinite(p).all() for p in P)


def test_training_steps_follow_the_definition():
    """Twenty steps with fresh gradients and carried momenta, of |P0 P1 - W|^2
    for a factored matrix: parameters and momenta after each, against the
    definition's step from the state and the gradients that it found
    (tests/test_oracle_muon.py: how far a step in a wrong direction or without
    its momentum would be off)."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda")
    W = draw(96, 16) @ draw(16, 64)
    grp = Group([(96, 16), (16, 64)], fresh=True)
    for p in grp.params:
        p.copy_(draw(*p.shape) * 0.1)
    P = grp.params
    for _ in range(20):
        R = P[0] @ P[1] - W
        grp.grads[0].copy_(R @ P[1].t())
        grp.grads[1].copy_(P[0].t() @ R)
        grp.keep()
        _srl().muon_step(grp.plan, 0.05)
        grp.check(0.05)


@pytest.mark.parametrize("rows,cols", [(256, 2097151), (2097151, 256), (3, 178956969), (536870911, 1)])
def test_largest_matrices(rows, cols):
    """Just below 2^29 elements, 2^31 bytes: against the definition in double,
    a stretch of the long side at a time."""
    import torch

    srl = _srl()
    s, L = min(rows, cols), max(rows, cols)
    gen = torch.Generator(device="cuda").manual_seed(rows % 1000)
    g = torch.randn((rows, cols), generator=gen, device="cuda")
    p, m = torch.zeros_like(g), torch.zeros_like(g)
    srl.muon_step(srl.muon_plan([p], [g], [m], lr_scale=[1.0]), 1.0, momentum=0.0)
    assert torch.equal(m, g)

    def pieces(x):
        x = x if rows <= cols else x.T
        each = (1 << 24) // s
        return (x[:, k:k + each].double().contiguous() for k in range(0, L, each))

    # (a library product over so long an axis with few rows takes seconds)
    square = lambda x: x @ x.T.contiguous() if s > 3 else (x[:, None] * x[None]).sum(2)
    gram, mags = (sum(square(f(x)) for x in pieces(g)) for f in (lambda x: x, torch.abs))
    norm = float(gram.diagonal().sum().sqrt()) + 1e-7
    sv, V = np.linalg.eigh((gram / norm ** 2).cpu().numpy())
    sv = np.maximum(sv, 0.0)
    q = om.growth(sv)
    Q = torch.from_numpy((V * q) @ V.T).cuda()
    # (as x_tolerance, for singular values far from zero: the slopes bound the quotients)
    lo, hi = sv.min() * 0.999, sv.max() * 1.001
    at = np.linspace(lo, hi, 20001)
    K = np.abs(np.diff(om.growth(at)) / np.diff(at)).max() * 1.01 * np.sqrt(hi)
    product = sum(float((Q.abs() @ (x.abs() / norm)).square().sum()) for x in pieces(g)) ** 0.5
    tol = (K * (4 * U * 16 * float(mags.norm()) / norm ** 2 + 6 * U) + 5 * U * float(Q.norm()) + 3 * U * np.abs(q).max()
           + 4 * U * 16 * product + 4 * U * s ** 0.5 * np.abs(q * np.sqrt(sv)).max())
    off = sum(float((y + Q @ (x / norm)).square().sum()) for x, y in zip(pieces(g), pieces(p))) ** 0.5
    say(f"  {rows} x {cols}: X off by {off:.2e}, allowed {tol:.2e}")
    assert off <= tol
    first, last = next(pieces(g)), (g if rows <= cols else g.T)[:, -5:].double()
    for x, y in ((first[:, :5], next(pieces(p))[:, :5]), (last, (p if rows <= cols else p.T)[:, -5:].double())):
        want = -(Q @ (x / norm))
        assert ((y - want).abs() <= 1e-4 * want.abs().max()).all()        # (at either end, each value of its own size)


def test_same_bits_every_time():
    import torch

    def once():
        grp = Group([(80, 1000), (999, 33), (200, 300)], seed=4)
        _srl().muon_step(grp.plan, 0.1)
        return grp.params + grp.st["m"]

    a = once()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, once()))


def test_nan_and_infinity_stay_in_their_matrix():
    import torch

    shapes = [(16, 300), (16, 300), (300, 80), (16, 300), (300, 80)]
    grp, ref = Group(shapes, seed=7), Group(shapes, seed=7)
    grp.grads[1][3, 200] = float("nan")
    grp.grads[2][1, 1] = float("inf")
    for x in (grp, ref):
        _srl().muon_step(x.plan, 0.1)
    for i in (0, 3, 4):
        assert torch.equal(grp.params[i], ref.params[i])
    for i in (1, 2):
        assert torch.isnan(grp.params[i]).all()


def test_matrices_end_where_they_end():
    """Matrices of odd sizes side by side in one buffer (16-byte starts): what
    lies between them stays."""
    import torch

    srl = _srl()
    shapes = [(13, 77), (77, 13), (81, 333), (1, 5), (97, 101), (129, 131)]
    room = [-(-r * c // 8) * 8 + 8 for r, c in shapes]
    views = lambda buf: [buf[a:a + r * c].view(r, c) for a, (r, c) in zip(np.cumsum([8] + room), shapes)]
    n = 8 + sum(room)
    for pt, gt, master in ((torch.float32, torch.float32, False), (torch.bfloat16, torch.bfloat16, True),
                           (torch.bfloat16, torch.float32, False)):
        bufs = [torch.full((n,), 3.0, dtype=t, device="cuda") for t in (pt, gt, torch.float32, torch.float32)]
        P, G, M, W = map(views, bufs)
        for g in G:
            g.copy_(torch.randn(g.shape, device="cuda"))
        plan = srl.muon_plan(P, G, M, master=W if master else None)
        srl.muon_step(plan, 0.1)
        hole = torch.ones(n, dtype=torch.bool, device="cuda")
        for h in views(hole):
            h.fill_(False)
        assert all((b[hole] == 3).all() for b in bufs)
        assert all(not (p == 3).all() for p in P)


def test_captured_step_with_dyn():
    import torch

    srl = _srl()
    a, b = (Group([(80, 640), (500, 24), (300, 150)], seed=8) for _ in range(2))
    dyn = torch.tensor([0.0, 1.0], device="cuda")
    srl.muon_step(a.plan, 0.0, dyn=dyn)              # (a zero rate moves the momenta alone)
    srl.muon_step(b.plan, 0.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        srl.muon_step(a.plan, 123.0, weight_decay=0.1, dyn=dyn)
    for lr, scale in ((0.1, 1.0), (0.02, 0.5), (0.3, 2.0)):
        dyn.copy_(torch.tensor([lr, scale]))
        torch.cuda.synchronize()
        graph.replay()
        srl.muon_step(b.plan, lr, weight_decay=0.1, grad_scale=scale)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.params + a.st["m"], b.params + b.st["m"]))
    with pytest.raises(srl.SalrError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            srl.muon_plan(a.params, a.grads, **a.st)


def test_step_on_another_stream():
    import torch

    srl = _srl()
    a, b = (Group([(80, 640), (500, 24)], seed=8) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    srl.muon_step(a.plan, 0.1, stream=s)
    s.synchronize()
    srl.muon_step(b.plan, 0.1)
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))


def test_refusals_of_the_binding():
    import torch

    srl = _srl()
    p = torch.zeros((16, 40), device="cuda")
    st = srl.muon_states([p])
    for bad in (dict(grads=[p.to(torch.float16)]), dict(grads=[p.t()]), dict(grads=[p[:8]]), dict(grads=[p.cpu()]),
                dict(params=[p.view(-1)]), dict(grads=[]), dict(master=[p, p]), dict(lr_scale=[1.0, 2.0])):
        with pytest.raises((TypeError, ValueError)):
            srl.muon_plan(**{**dict(params=[p], grads=[p.clone()], m=st["m"]), **bad})
    with pytest.raises(srl.SalrError):
        srl.muon_plan([p], [p], st["m"])                                  # the gradient is what is written
    with pytest.raises(srl.SalrError):
        srl.muon_plan([p], [p.clone()], st["m"], master=[p.clone()])      # a master of a float parameter
    big = torch.zeros((257, 300), device="cuda")
    with pytest.raises(srl.SalrError):
        srl.muon_plan([big], [big.clone()], srl.muon_states([big])["m"])
    plan = srl.muon_plan([p], [p.clone()], st["m"])
    for bad in (dict(lr=-1.0), dict(momentum=1.0), dict(eps=0.0), dict(steps=0), dict(steps=7),
                dict(coefficients=(1.0, float("nan"), 0.0)), dict(grad_scale=float("inf"))):
        with pytest.raises(srl.SalrError):
            srl.muon_step(plan, **{**dict(lr=0.1), **bad})
