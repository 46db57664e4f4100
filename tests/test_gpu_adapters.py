"""The adapters of many requests on the GPU against the float64 oracle
(oracle/adapters.py).

Tolerances, derived: u = 2^-24 is fp32's half step, h = 2^-8 bf16's.
 - T, G: n products of bf16 values (exact in fp32) summed in fp32 in any
   order: (n + 64) u of the sum of magnitudes; times the scale: u more.
 - met by the next product as two bf16 values: what is left of the first
   rounding is at most h of the value, of the second h^2 = 2^-16; as three
   (gradients): 2^-24.
 - Y, dX: those errors times the weights' magnitudes, 2 r + 8 sums of u of
   the sum of magnitudes, and h of the result.
 - dA, dB: those of G and T times the columns' magnitudes, 3 M + 64 sums of u
   of the sum of magnitudes.
Copies of base, zeros and the plan's indexes are exact."""

import numpy as np
import pytest

from oracle import adapters as oa
from oracle import bf16 as ob
from tests.gpu_util import say, to_dev, to_host_bits

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
NAN = float("nan")


def _srl():
    import sparse_rank_linear_amd as srl

    return srl


def _bf16(x):
    bits = ob.f64_to_bits(np.asarray(x, dtype=np.float64))
    return ob.bits_to_f64(bits), bits


class Case:
    """Inputs of one call, as float64 and on the device."""

    def __init__(self, M, count, r, K, N, ids="runs", mixed=True, base=True, seed=0):
        import torch

        g = np.random.default_rng(seed)
        self.M, self.count, self.r, self.K, self.N = M, count, r, K, N
        draw = lambda scale, *s: _bf16(g.standard_normal(s) * scale)
        (self.a, ab), (self.b, bb) = draw(0.3, count, r, K), draw(0.3, count, N, r)
        (self.X, xb), (self.dY, yb) = draw(1.0, M, K), draw(1.0, M, N)
        (self.by, byb), (self.bx, bxb) = draw(2.0, M, N), draw(2.0, M, K)
        if ids == "runs":            # requests of ragged lengths, some without an adapter
            cuts = np.sort(g.integers(0, M + 1, max(0, min(M, 2 * count) - 1)))
            self.ids = (np.searchsorted(cuts, np.arange(M), side="right") * 7 + 1) % (count + 1)
            self.ids[self.ids == count] = -1
        elif ids == "random":        # any values
            self.ids = g.integers(-2, count + 2, M)
            self.ids[::17] = 2 ** 31 - 1
            self.ids[1::19] = -2 ** 31
        else:
            self.ids = np.full(M, ids)
        self.ranks = np.array([max(0, r - 5 * q) if mixed else r for q in range(count)])
        self.scales = np.where(np.arange(count) % 3 == 2, -0.75, 1.0 + 0.25 * np.arange(count)) if mixed else np.ones(
            count)
        if mixed and count > 2:
            self.ranks[2] = 0        # an adapter that is not there yet
        if mixed:                    # what is not used may be anything
            ab, bb, xb = ab.copy(), bb.copy(), xb.copy()
            for q in range(count):
                ab[q, self.ranks[q]:] = 0x7FC0
                bb[q, :, self.ranks[q]:] = 0x7FC0
            bare = (self.ids < 0) | (self.ids >= count)
            xb[bare] = 0x7FC0
            yb = yb.copy()
            yb[bare] = 0x7FC0
        if not base:
            self.by, self.bx = np.zeros((M, N)), np.zeros((M, K))
        up = lambda b: to_dev(b)
        self.ids_d = torch.from_numpy(self.ids.astype(np.int32)).cuda()
        self.ad = _srl().SalrAdapters(
            up(ab), up(bb), ranks=torch.from_numpy(self.ranks.astype(np.int32)).cuda() if mixed else None,
            scales=torch.from_numpy(self.scales.astype(np.float32)).cuda() if mixed else None)
        self.X_d, self.dY_d = up(xb), up(yb)
        self.by_d, self.bx_d = (up(byb), up(bxb)) if base else (None, None)
        self.scales = self.scales.astype(np.float32).astype(np.float64)

    def _magnitudes(self):
        """Per token: the oracle's inputs as magnitudes."""
        return np.abs(self.a), np.abs(self.b), np.abs(self.scales)

    def check_forward(self, Y):
        want = oa.forward(self.a, self.b, self.ids, self.ranks, self.scales, self.X, self.by)
        A, B, S = self._magnitudes()
        tol = np.abs(want) * H + 1e-37
        for t, q in oa._tokens(self.ids, self.count):
            n = self.ranks[q]
            T, mag = np.abs(self.a[q, :n] @ self.X[t]) * S[q], (A[q, :n] @ np.abs(self.X[t])) * S[q]
            err = (self.K + 64) * U * mag + (2 * U + 2.0 ** -16) * T
            tol[t] += (1 + H) * (B[q, :, :n] @ err + (2 * self.r + 8) * U * (B[q, :, :n] @ mag))
        got = ob.bits_to_f64(to_host_bits(Y))
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], tol[bad][:4])
        bare = np.array([not (0 <= q < self.count) or self.ranks[q] == 0 for q in self.ids], dtype=bool)
        assert (got[bare] == self.by[bare]).all()

    def check_backward(self, dX, dA, dB):
        wx, wa, wb = oa.backward(self.a, self.b, self.ids, self.ranks, self.scales, self.X, self.dY, self.bx)
        A, B, S = self._magnitudes()
        tx, ta, tb = np.abs(wx) * H + 1e-37, np.zeros(wa.shape), np.zeros(wb.shape)
        sums = (3 * self.M + 64) * U
        for t, q in oa._tokens(self.ids, self.count):
            n, x, y = self.ranks[q], np.abs(self.X[t]), np.abs(self.dY[t])
            T, mt = np.abs(self.a[q, :n] @ self.X[t]) * S[q], (A[q, :n] @ x) * S[q]
            G, mg = np.abs(self.dY[t] @ self.b[q, :, :n]) * S[q], (y @ B[q, :, :n]) * S[q]
            et, eg = ((k + 64) * U * m + 2 * U * v for k, m, v in ((self.K, mt, T), (self.N, mg, G)))
            tx[t] += (1 + H) * ((eg + 2.0 ** -16 * G) @ A[q, :n] + (2 * self.r + 8) * U * (mg @ A[q, :n]))
            ta[q, :n] += np.outer(eg + 2.0 ** -24 * G + sums * G, x)
            tb[q, :, :n] += np.outer(y, et + 2.0 ** -24 * T + sums * T)
        for name, got, want, tol in (("dX", None if dX is None else ob.bits_to_f64(to_host_bits(dX)), wx, tx),
                                     ("dA", dA.double().cpu().numpy(), wa, ta),
                                     ("dB", dB.double().cpu().numpy(), wb, tb)):
            if got is None:
                continue
            bad = ~(np.abs(got - want) <= tol)
            assert not bad.any(), (name, np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], tol[bad][:4])


# M, count, r, K, N, ids: one token, tiles of 16 and 64 tokens and around them,
# columns in eights around 64 and 256, odd outputs, one adapter and very many
FORWARD = [(1, 1, 8, 8, 1, 0), (1, 3, 16, 264, 40, 1), (5, 2, 16, 512, 72, "random"), (16, 1, 16, 4096, 64, 0),
           (17, 4, 24, 136, 65, "random"), (33, 5, 32, 72, 256, "random"), (63, 1, 40, 256, 7, 0),
           (64, 3, 64, 320, 130, "runs"), (65, 2, 80, 200, 264, 1), (129, 7, 96, 1032, 96, "runs"),
           (200, 70, 112, 96, 33, "random"), (300, 4, 128, 128, 1030, "runs"), (90, 3, 160, 264, 48, "runs"),
           (70, 2, 256, 520, 520, "random"), (1500, 6, 16, 64, 24, "runs"), (40, 4096, 8, 16, 8, "random"),
           (3, 2, 16, 14344, 16, "random"), (12, 3, 8, 64, 4100, "runs")]


@pytest.mark.parametrize("M,count,r,K,N,ids", FORWARD)
def test_plan_and_forward(M, count, r, K, N, ids):
    srl = _srl()
    c = Case(M, count, r, K, N, ids, seed=M + r)
    plan = srl.adapters_plan(c.ids_d, count)
    say("forward", M, count, r, K, N, ids)
    c.check_forward(srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d))


BACKWARD = [(1, 1, 8, 8, 8, 0), (1, 3, 16, 264, 40, 1), (5, 2, 16, 512, 72, "random"), (17, 4, 24, 136, 64, "random"),
            (33, 5, 32, 72, 256, "random"), (63, 1, 40, 256, 8, 0), (64, 3, 64, 320, 136, "runs"),
            (65, 2, 80, 200, 264, 1), (129, 7, 96, 1032, 96, "runs"), (200, 70, 112, 96, 32, "random"),
            (90, 3, 160, 264, 48, "runs"), (70, 2, 256, 136, 264, "random"), (1500, 6, 16, 64, 24, "runs"),
            (2500, 2, 8, 16, 8, "runs"), (1024, 1, 16, 8, 16, 0), (1025, 1, 16, 16, 8, 0), (40, 2048, 8, 16, 8, "random")]


@pytest.mark.parametrize("M,count,r,K,N,ids", BACKWARD)
def test_backward(M, count, r, K, N, ids):
    srl = _srl()
    c = Case(M, count, r, K, N, ids, seed=M + r)
    plan = srl.adapters_plan(c.ids_d, count)
    say("backward", M, count, r, K, N, ids)
    c.check_backward(*srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, base=c.bx_d))


def _plan_arrays(plan, count):
    """(offsets, order) out of a plan's buffer (after a 16-byte head; arrays
    from multiples of 16 bytes)."""
    w = plan.buffer.cpu().numpy().view(np.int32)
    n, M = count + 2, plan.M
    skip = -(-n // 4) * 4
    return w[4:4 + n], w[4 + 2 * skip:4 + 2 * skip + M]


@pytest.mark.parametrize("M,count", [(0, 1), (1, 1), (63, 5), (64, 1), (1000, 3), (1024, 1024), (1025, 2000), (1000, 1025), (5000, 4096),
                                     (70000, 17)])
def test_plan_order(M, count):
    import torch

    srl = _srl()
    ids = np.random.default_rng(M).integers(-1, count + 1, M).astype(np.int32)
    plan = srl.adapters_plan(torch.from_numpy(ids).cuda(), count)
    off, order = _plan_arrays(plan, count)
    g = np.where((ids >= 0) & (ids < count), ids, count)
    np.testing.assert_array_equal(order, np.argsort(g, kind="stable"))
    np.testing.assert_array_equal(off, np.concatenate([np.searchsorted(np.sort(g), np.arange(count + 1)), [M]]))
    if M <= 1025:
        want = oa.plan(ids, count)
        np.testing.assert_array_equal(off, want[0])
        np.testing.assert_array_equal(order, want[1])


def _zeros_like_guarded(shape, dtype, guard=512):
    """A tensor of `shape` inside a buffer whose ends hold a pattern, and a check of them."""
    import torch

    n = int(np.prod(shape))
    buf = torch.full((n + 2 * guard,), 7.0, dtype=dtype, device="cuda")
    t = buf[guard:guard + n].view(shape)
    return t, lambda: bool((buf[:guard] == 7).all()) and bool((buf[guard + n:] == 7).all())


def test_outputs_end_where_they_end():
    import torch

    srl = _srl()
    c = Case(77, 3, 24, 136, 72, "random", seed=5)
    Y, y_ok = _zeros_like_guarded((77, 72), torch.bfloat16)
    dX, x_ok = _zeros_like_guarded((77, 136), torch.bfloat16)
    dA, a_ok = _zeros_like_guarded((3, 24, 136), torch.float32)
    dB, b_ok = _zeros_like_guarded((3, 72, 24), torch.float32)
    ws, w_ok = _zeros_like_guarded((srl.adapters_ws_bytes(3, 72, 136, 24, 77, True),), torch.uint8)
    plan = srl.adapters_plan(c.ids_d, 3)
    c.check_forward(srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d, Y=Y, ws=ws))
    c.check_backward(*srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, base=c.bx_d, dX=dX, dA=dA, dB=dB, ws=ws))
    assert y_ok() and x_ok() and a_ok() and b_ok() and w_ok()


@pytest.mark.parametrize("M", [9, 70, 1300])
def test_base_in_place_none_and_skipped_dx(M):
    srl = _srl()
    c = Case(M, 3, 16, 72, 40, "runs", seed=M)
    plan = srl.adapters_plan(c.ids_d, 3)
    want = srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d)
    Y = c.by_d.clone()
    assert srl.adapters_forward(c.ad, plan, c.X_d, base=Y, Y=Y) is Y and (Y == want).all()
    dx, da, db = srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, base=c.bx_d)
    none, da2, db2 = srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, need_dx=False)
    assert none is None and (da2 == da).all() and (db2 == db).all()
    x = c.bx_d.clone()
    assert (srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, base=x, dX=x)[0] == dx).all()
    z = Case(M, 3, 16, 72, 40, "runs", base=False, seed=M)
    z.check_forward(srl.adapters_forward(z.ad, plan, z.X_d))
    z.check_backward(*srl.adapters_backward(z.ad, plan, z.X_d, z.dY_d))


def test_a_buffer_serves_shorter_batches():
    """A plan of 1100 tokens, whose tiles are large, used again for 1000, whose
    tiles are small and more."""
    import torch

    srl = _srl()
    plan = srl.adapters_plan(torch.zeros(1100, dtype=torch.int32, device="cuda"), 300)
    c = Case(1000, 300, 8, 16, 8, "random", seed=2)
    assert srl.adapters_plan(c.ids_d, 300, plan=plan) is plan
    c.check_forward(srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d))


def test_replaced_tensors_and_memory():
    """What the adapters hold when a call is made is what it uses, though a
    tensor, or the memory behind one, has been replaced since the last."""
    srl = _srl()
    c, d = (Case(40, 4, 16, 72, 48, "runs", mixed=False, seed=q) for q in (3, 3))
    for q in (0, 1):
        plan = srl.adapters_plan(c.ids_d, 4)
        c.check_forward(srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d))
        keep = c.ad.a.data, c.ad.b.data        # (alive: the new memory is elsewhere)
        if q == 0:
            c.ad.a.data, c.ad.b.data = d.ad.a.flip(0), d.ad.b.flip(0)
        else:
            c.ad.a, c.ad.b = d.ad.a.flip(0), d.ad.b.flip(0)
            c.a, c.b = d.a, d.b
        c.a, c.b = c.a[::-1], c.b[::-1]
        c.check_forward(srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d))
        del keep
    c.ad.b.data = d.ad.b[:3].clone()
    with pytest.raises(ValueError):
        srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d)


def test_shrunk_at_the_same_address():
    """Fewer adapters in the memory of more: the calls work on, and write the
    gradients of, as many as there are now."""
    import torch

    srl = _srl()
    c = Case(90, 4, 24, 136, 72, "runs", seed=6)
    plan = srl.adapters_plan(c.ids_d, 4)
    c.check_forward(srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d))
    for t in (c.ad.a, c.ad.b, c.ad.ranks, c.ad.scales):
        t.data = t.data[:2]
    c.count, c.a, c.b, c.ranks, c.scales = 2, c.a[:2], c.b[:2], c.ranks[:2], c.scales[:2]
    with pytest.raises(srl.SalrError):                                   # (a plan of four)
        srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d)
    srl.adapters_plan(c.ids_d, 2, plan=plan)
    c.check_forward(srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d))
    dA, a_ok = _zeros_like_guarded((2, 24, 136), torch.float32, 4 * 24 * 136)
    dB, b_ok = _zeros_like_guarded((2, 72, 24), torch.float32, 4 * 24 * 136)
    c.check_backward(*srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, base=c.bx_d, dA=dA, dB=dB))
    assert a_ok() and b_ok()
    got = srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, need_dx=False)[1:]
    assert torch.equal(got[0], dA) and torch.equal(got[1], dB)


def test_no_tokens():
    import torch

    srl = _srl()
    ad = srl.SalrAdapters.empty(2, 16, 24, 8)
    plan = srl.adapters_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 2)
    X = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    dY = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    assert srl.adapters_forward(ad, plan, X).shape == (0, 16)
    dA, dB = (torch.ones(s, device="cuda") for s in (ad.a.shape, ad.b.shape))
    srl.adapters_backward(ad, plan, X, dY, dA=dA, dB=dB)
    assert (dA == 0).all() and (dB == 0).all()


def test_infinite_values_reach_their_own_outputs_only():
    """An infinite product is an infinite output (its bf16 parts are not inf -
    inf), and only its token's."""
    import torch

    srl = _srl()
    a = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device="cuda")
    a[0, 0, 0] = 1.0
    b = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device="cuda")
    b[0, :, 0] = 2.0
    X = torch.ones((20, 8), dtype=torch.bfloat16, device="cuda")
    X[3, 0] = float("inf")
    X[7, 0] = NAN
    plan = srl.adapters_plan(torch.zeros(20, dtype=torch.int32, device="cuda"), 1)
    Y = srl.adapters_forward(srl.SalrAdapters(a, b), plan, X).float()
    # (0 * inf of the other ranks is NaN by the formula where b's row has them; here rank 0 alone counts)
    assert torch.isnan(Y[7]).all() and not torch.isfinite(Y[3]).any()
    assert (Y[[t for t in range(20) if t not in (3, 7)]] == 2.0).all()


class NotFinite:
    """A backward call with one value of X or dY infinite or NaN, beside the
    same call with zero there (checked against the oracle): adapters of
    `ranks` ranks, the value in a token of the middle one."""

    def __init__(self, M, r, ranks, where, value, fresh=False):
        import torch

        srl = _srl()
        c = Case(M, len(ranks), r, 136, 72, "runs", mixed=False, seed=M + r)
        c.ranks = np.array(ranks)
        if fresh:                    # the first rank of A and B zeros
            for x in (c.a, c.ad.a):
                x[:, 0] = 0.0
            for x in (c.b, c.ad.b):
                x[:, :, 0] = 0.0
        c.ad.ranks = torch.tensor(ranks, dtype=torch.int32, device="cuda")
        plan = srl.adapters_plan(c.ids_d, len(ranks))
        mine = np.flatnonzero(c.ids == len(ranks) // 2)
        at = (int(mine[2 * len(mine) // 3]), 41)
        host, dev = (c.X, c.X_d) if where == "X" else (c.dY, c.dY_d)
        call = lambda: srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, base=c.bx_d)
        host[at] = dev[at] = 0.0
        clean = call()
        c.check_backward(*clean)
        host[at] = dev[at] = value
        got = call()
        with np.errstate(invalid="ignore"):
            self.want = oa.backward(c.a, c.b, c.ids, c.ranks, c.scales, c.X, c.dY, c.bx)
        self.got, self.clean = ([t.double().cpu().numpy() for t in x] for x in (got, clean))
        self.ranks = ranks


NOT_FINITE = [(M, r, ranks, where, value) for M, r, ranks in ((200, 32, (24, 5, 12)), (200, 32, (5, 24, 12)),
                                                             (4000, 32, (24, 12, 5)), (3000, 96, (5, 85, 90)))
              for where in ("X", "dY") for value in (float("inf"), -float("inf"), NAN)]


@pytest.mark.parametrize("M,r,ranks,where,value", NOT_FINITE)
def test_unused_ranks_get_zeros_beside_values_that_are_not_finite(M, r, ranks, where, value):
    """One chunk of an adapter's tokens, and several.  What the formula gives
    as finite is what the call without that value gives, to the bit."""
    q = NotFinite(M, r, ranks, where, value)
    for i, n in enumerate(ranks):
        assert (q.got[1][i, n:] == 0).all() and (q.got[2][i, :, n:] == 0).all()
    for name, got, want, clean in zip(("dX", "dA", "dB"), q.got, q.want, q.clean):
        finite = np.isfinite(want)
        assert (np.isfinite(got) == finite).all(), name
        assert (got[finite] == clean[finite]).all(), name
    assert not np.isfinite(q.want[1]).all() and not np.isfinite(q.want[2]).all()


@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("M,r,ranks,where,value", NOT_FINITE)
def test_gradients_of_infinite_values_follow_the_formula(M, r, ranks, where, value, fresh):
    """Infinite, with its sign, where the formula is, and NaN where it is."""
    q = NotFinite(M, r, ranks, where, value, fresh)
    for name, got, want in zip(("dX", "dA", "dB"), q.got, q.want):
        bad = ~np.isfinite(want) & ~((got == want) | (np.isnan(got) & np.isnan(want)))
        assert not bad.any(), (name, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), NAN])
@pytest.mark.parametrize("M,r", [(1, 8), (200, 40), (3000, 96)])
def test_outputs_of_infinite_values_follow_the_formula(M, r, value):
    """One value of X, then one of the base as well: what the formula gives, and
    other tokens as without them."""
    srl = _srl()
    c = Case(M, 2, r, 136, 72, M % 2, mixed=False, seed=M)
    plan = srl.adapters_plan(c.ids_d, 2)
    c.X[M // 2, 77] = c.X_d[M // 2, 77] = 0.0
    clean = srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d)
    c.check_forward(clean)
    for base in (False, True):
        c.X[M // 2, 77] = c.X_d[M // 2, 77] = value
        if base:
            c.by[M // 2, 5] = c.by_d[M // 2, 5] = float("inf")
        got = srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d).double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            want = oa.forward(c.a, c.b, c.ids, c.ranks, c.scales, c.X, c.by)
        assert not np.isfinite(want[M // 2]).any()
        np.testing.assert_array_equal(got[M // 2], want[M // 2])
        others = np.arange(M) != M // 2
        assert (got[others] == clean.double().cpu().numpy()[others]).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("M", [1, 1100])
def test_sums_that_bf16_would_round_to_infinity(M, sign):
    """T (and G) of 2^128 - 2^119 + 2^112: a float holds it, its nearest bf16
    would be infinite."""
    import torch

    srl = _srl()
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    plan = srl.adapters_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), 1)
    big, rest = sign * (2.0 ** 128 - 2.0 ** 120), sign * (2.0 ** 119 + 2.0 ** 112)
    a, b, X, dY = z(1, 8, 72), z(1, 72, 8), z(M, 72), z(M, 72)
    a[0, 0, 3] = a[0, 0, 40] = 1.0
    b[0, 5, 0] = 2.0 ** -10
    X[:, 3], X[:, 40] = big, rest
    dY[0, 7] = 2.0 ** -10
    ad = srl.SalrAdapters(a, b)
    Y = srl.adapters_forward(ad, plan, X)
    assert (Y[:, 5] == sign * 2.0 ** 118).all() and Y.count_nonzero() == M
    dB = srl.adapters_backward(ad, plan, X, dY)[2]
    assert dB[0, 7, 0].item() == (big + rest) * 2.0 ** -10 and dB.count_nonzero() == 1
    # the other way round: G
    ad = srl.SalrAdapters(b.transpose(1, 2).contiguous(), a.transpose(1, 2).contiguous())
    dX, dA, _ = srl.adapters_backward(ad, plan, dY, X)
    assert (dX[:, 5] == sign * 2.0 ** 118).all() and dX.count_nonzero() == M
    assert dA[0, 0, 7].item() == (big + rest) * 2.0 ** -10 and dA.count_nonzero() == 1


@pytest.mark.parametrize("M", [40, 1500])
def test_same_bits_every_time_and_any_workspace(M):
    """Results do not depend on timing, on what the workspace held, or on the
    plan's buffer being one of a longer batch."""
    import torch

    srl = _srl()
    c = Case(M, 5, 40, 264, 136, "runs", seed=M)
    plan = srl.adapters_plan(torch.zeros(2 * M, dtype=torch.int32, device="cuda"), 5)
    srl.adapters_plan(c.ids_d, 5, plan=plan)
    ws = srl.adapters_workspace(c.ad, 2 * M, backward=True)
    first = None
    for fill in (0, 255, 127):
        ws.fill_(fill)
        got = [srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d, ws=ws),
               *srl.adapters_backward(c.ad, plan, c.X_d, c.dY_d, base=c.bx_d, ws=ws)]
        first = first or got
        assert all((x == y).all() for x, y in zip(first, got))
    c.check_forward(first[0])
    c.check_backward(*first[1:])


@pytest.mark.parametrize("M,r,K,N,backward", [(140000, 40, 512, 16, True), (140000, 40, 16, 512, True),
                                              (70000, 16, 512, 16, True), (5000, 88, 1024, 64, True),
                                              (1025, 40, 8192, 16, True), (1024, 256, 4096, 16, True),
                                              (90000, 64, 1024, 8, False), (1025, 256, 8192, 8, False)])
def test_workspace_ends_where_it_ends(M, r, K, N, backward):
    """One side much longer than the other, few and many tiles: nothing is
    written behind the workspace, and the pieces make the product."""
    import torch

    srl = _srl()
    g = torch.Generator(device="cuda").manual_seed(M + r)
    draw = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    ad = srl.SalrAdapters(draw(2, r, K), draw(2, N, r))
    X, dY = draw(M, K), draw(M, N)
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % 2
    plan = srl.adapters_plan(ids, 2)
    need = srl.adapters_ws_bytes(2, N, K, r, M, backward)
    buf = torch.full((need + (64 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[:need]
    d = lambda t: t.double()
    if backward:
        dX, dA, dB = srl.adapters_backward(ad, plan, X, dY, ws=ws)
    else:
        Y = srl.adapters_forward(ad, plan, X, ws=ws)
    assert (buf[need:] == 0xA5).all()
    for q in (0, 1):
        x, y, A, B = d(X[q::2]), d(dY[q::2]), d(ad.a[q]), d(ad.b[q])
        if not backward:
            got, want, left, right = Y[q::2], x @ A.T.contiguous() @ B.T.contiguous(), x @ A.T.contiguous(), B
            size = x.abs() @ A.abs().T.contiguous() @ B.abs().T.contiguous()
            tol = want.abs() * H + ((K + r + 64) * U) * size + 2.0 ** -16 * (left.abs() @ right.abs().T.contiguous())
            assert ((d(got) - want).abs() <= tol * 1.1).all()
            continue
        G, T = y @ B, x @ A.T.contiguous()
        mag = y.abs() @ B.abs() @ A.abs()
        tol = (G @ A).abs() * H + (N + r + 64) * U * mag + 2.0 ** -16 * (G.abs() @ A.abs())
        assert ((d(dX[q::2]) - G @ A).abs() <= tol * 1.1).all()
        # (sums of M / 2 products of either side, whose own sums are K or N long)
        t = lambda v: v.T.contiguous()
        bound = (3 * (M // 2) + K + N + 64) * U
        assert ((d(dA[q]) - t(G) @ x).abs() <= bound * (t(y.abs() @ B.abs()) @ x.abs())).all()
        assert ((d(dB[q]) - t(y) @ T).abs() <= bound * (t(y.abs()) @ (x.abs() @ t(A.abs())))).all()


def test_captured_batches_with_other_ids():
    """Plan, forward and backward captured once: each replay takes the ids and
    inputs it finds."""
    import torch

    srl = _srl()
    cases = [Case(M, 4, 24, 136, 72, "random", seed=s) for s, M in ((1, 90), (2, 90), (3, 90))]
    c = cases[0]
    ids, X, dY = c.ids_d.clone(), c.X_d.clone(), c.dY_d.clone()
    ws = srl.adapters_workspace(c.ad, 90, backward=True)
    plan = srl.adapters_plan(ids, 4)
    Y, dX = torch.empty_like(c.by_d), torch.empty_like(c.bx_d)
    dA, dB = torch.empty(c.ad.a.shape, device="cuda"), torch.empty(c.ad.b.shape, device="cuda")

    def call():
        srl.adapters_plan(ids, 4, plan=plan)
        srl.adapters_forward(c.ad, plan, X, Y=Y, ws=ws)
        srl.adapters_backward(c.ad, plan, X, dY, dX=dX, dA=dA, dB=dB, ws=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for q in (1, 2, 0, 1):
        for dst, src in ((ids, cases[q].ids_d), (X, cases[q].X_d), (dY, cases[q].dY_d)):
            dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        p2 = srl.adapters_plan(cases[q].ids_d, 4)
        want = [srl.adapters_forward(c.ad, p2, X), *srl.adapters_backward(c.ad, p2, X, dY)]
        # (tokens without an adapter hold NaN inputs: their outputs are zeros)
        assert all((x == y).all() for x, y in zip((Y, dX, dA, dB), want))


def test_two_streams_with_their_own_workspaces():
    import torch

    srl = _srl()
    c = Case(1200, 6, 32, 520, 264, "runs", seed=9)
    plan = srl.adapters_plan(c.ids_d, 6)
    want = srl.adapters_forward(c.ad, plan, c.X_d, base=c.by_d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            p = srl.adapters_plan(c.ids_d, 6, stream=s)
            got.append(srl.adapters_forward(c.ad, p, c.X_d, base=c.by_d, stream=s))
    torch.cuda.synchronize()
    assert all((g == want).all() for g in got)


def test_offsets_past_32_bits():
    """X of more than 2^32 bytes and elements past 2^31."""
    import torch

    srl = _srl()
    M, K, N, r = 270000, 8192, 8, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    ad = srl.SalrAdapters((torch.randn((2, r, K), generator=g, device="cuda") * 0.1).to(torch.bfloat16),
                          torch.randn((2, N, r), generator=g, device="cuda").to(torch.bfloat16))
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 131071, 262143, 262145, M - 2, M - 1], device="cuda")
    X[at] = torch.randn((len(at), K), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % 3          # (2: no adapter)
    Y = srl.adapters_forward(ad, srl.adapters_plan(ids, 2), X)
    some = torch.zeros(M, dtype=torch.bool, device="cuda")
    some[at] = True
    assert (Y[~some] == 0).all()
    for t in at.tolist():
        q = t % 3
        if q == 2:
            assert (Y[t] == 0).all()
            continue
        x, A, B = (v.double() for v in (X[t], ad.a[q], ad.b[q]))
        T = A @ x
        tol = (B.abs() @ ((K + 64) * U * (A.abs() @ x.abs()) + 2.0 ** -16 * T.abs())) * 1.1 + (B @ T).abs() * H
        assert ((Y[t].double() - B @ T).abs() <= tol).all()


def test_refusals_of_the_binding():
    import torch

    srl = _srl()
    ad = srl.SalrAdapters.empty(2, 16, 24, 8)
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    plan = srl.adapters_plan(ids, 2)
    X = torch.zeros((5, 24), dtype=torch.bfloat16, device="cuda")
    for bad in (X.float(), X[:4], X.cpu(), torch.zeros((24, 5), dtype=torch.bfloat16, device="cuda").t()):
        with pytest.raises((TypeError, ValueError)):
            srl.adapters_forward(ad, plan, bad)
    with pytest.raises(srl.SalrError):
        srl.adapters_forward(ad, srl.adapters_plan(ids, 3), X)           # a plan of other adapters
    with pytest.raises(srl.SalrError):
        srl.adapters_forward(ad, plan, X, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(srl.SalrError):
        srl.adapters_plan(torch.zeros(5000, dtype=torch.int32, device="cuda"), 2, plan=plan)   # a longer batch
    with pytest.raises(ValueError):
        srl.SalrAdapters(ad.a, ad.b[:1])
    with pytest.raises(TypeError):
        srl.adapters_plan(ids.long(), 2)
    assert plan.M == 5                                                    # (as it was)
    assert (srl.adapters_forward(ad, plan, X) == 0).all()
