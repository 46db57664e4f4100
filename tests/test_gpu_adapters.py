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
