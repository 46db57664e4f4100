"""How many bits of X A and of G the adapters' second products see: cases in
which all sums are exact, so that results are known to the bit.

A token's T (or G) is s (m1 + m2 2^-8 + m3 2^-16) 2^e with whole m of 128 to 255
and a power of two s: 24 bits, which a float holds.  What meets it has one value
a token, a power of two, where no other token has one: every gradient element
is one product, 24 bits, and zeros.  T of m1 + m2 2^-8 alone (16 bits), against
a base of minus its first bf16 part, leaves m2 2^-8 or what is missing of it: 8
bits, which bf16 holds."""

import numpy as np
import pytest

from oracle import adapters as oa
from oracle import bf16 as ob
from tests.gpu_util import to_dev, to_host_bits

LONG, AT = 136, (3, 40, 100)     # the columns of the exact sums: in different products of 32


def _whole(g, *shape):
    return g.integers(128, 256, shape).astype(np.float64)


def parts(x, n):
    """x as the sum of its first n bf16 parts."""
    got = np.zeros_like(x)
    for _ in range(n):
        got = got + ob.bits_to_f64(ob.f64_to_bits(x - got))
    return got


class Exact:
    """M tokens of two adapters of rank r.  side "a": G holds 24 bits, for dA;
    side "b": T, for dB."""

    def __init__(self, M, r, side, seed=0):
        g = np.random.default_rng(seed + M + r)
        self.side, self.ids, self.scales = side, np.arange(M) % 2, np.array([1.0, 0.5])
        self.ranks = np.array([r, max(1, r - 3)])
        short = -(-M // 8) * 8
        digits, one = np.zeros((M, LONG)), np.zeros((M, short))
        digits[:, AT] = np.array([1.0, 2.0 ** -8, 2.0 ** -16]) * 2.0 ** (np.arange(M) % 5 - 2.0)[:, None]
        one[np.arange(M), np.arange(M)] = 2.0 ** (np.arange(M) % 7 - 3.0) * (1 - 2 * (np.arange(M) % 2))
        weights, other = _whole(g, 2, r, LONG), _whole(g, 2, r, short)
        rows = lambda w: np.ascontiguousarray(w.transpose(0, 2, 1))
        if side == "a":
            self.X, self.dY, self.a, self.b = one, digits, other, rows(weights)
        else:
            self.X, self.dY, self.a, self.b = digits, one, weights, rows(other)
        self.base = np.zeros(self.X.shape)

    def want(self, n_parts=None):
        """(dA or dB) by the oracle; n_parts: from so many bf16 parts of G and T."""
        if n_parts is None:
            return oa.backward(self.a, self.b, self.ids, self.ranks, self.scales, self.X, self.dY, self.base)[
                1 if self.side == "a" else 2]
        out = np.zeros(self.a.shape if self.side == "a" else self.b.shape)
        for t, q in enumerate(self.ids):
            n = self.ranks[q]
            if self.side == "a":
                out[q, :n] += np.outer(parts(self.scales[q] * (self.dY[t] @ self.b[q, :, :n]), n_parts), self.X[t])
            else:
                out[q, :, :n] += np.outer(self.dY[t], parts(self.scales[q] * (self.a[q, :n] @ self.X[t]), n_parts))
        return out


class Small:
    """M tokens whose T (side "Y") or G (side "dX") holds 16 bits, written out
    by weights of a single one an output, onto a base that takes the first
    part away."""

    def __init__(self, M, r, side, seed=0):
        g = np.random.default_rng(seed + M + r)
        self.side, self.ids, self.scales = side, np.arange(M) % 2, np.array([1.0, 2.0])
        self.ranks = np.array([r, r])
        digits = np.zeros((M, LONG))
        digits[:, AT[:2]] = np.array([1.0, 2.0 ** -8])
        weights, out = _whole(g, 2, r, LONG), 2 * r
        ones = np.zeros((2, r, out))
        ones[:, np.arange(out) % r, np.arange(out)] = 1.0
        rows = lambda w: np.ascontiguousarray(w.transpose(0, 2, 1))
        if side == "Y":
            self.X, self.a, self.b, self.dY = digits, weights, rows(ones), None
        else:
            self.dY, self.b, self.a, self.X = digits, rows(weights), ones, np.zeros((M, out))
        t = np.stack([self.scales[q] * (weights[q] @ digits[i]) for i, q in enumerate(self.ids)])
        self.t, self.base = t[:, np.arange(out) % r], -parts(t, 1)[:, np.arange(out) % r]

    def want(self, n_parts=None):
        if n_parts is not None:
            return self.base + parts(self.t, n_parts)
        if self.side == "Y":
            return oa.forward(self.a, self.b, self.ids, self.ranks, self.scales, self.X, self.base)
        return oa.backward(self.a, self.b, self.ids, self.ranks, self.scales, self.X, self.dY, self.base)[0]


def _bits(x):
    b = ob.f64_to_bits(x)
    assert (ob.bits_to_f64(b) == x).all()          # (a bf16 value as it is)
    return b


# few and many tokens, a second stage of 32, several chunks; rank tiles and
# groups of them
SIZES = [(1, 8), (1, 96), (70, 8), (70, 40), (200, 88), (1300, 16), (1100, 40), (1100, 96)]


@pytest.mark.parametrize("M,r", SIZES[:6])
def test_the_cases_tell_the_parts_apart(M, r):
    """On the CPU: three parts are all of a value, two or one are not."""
    for side in ("a", "b"):
        c = Exact(M, r, side)
        want = c.want()
        assert (want == want.astype(np.float32)).all() and (c.want(3) == want).all()
        for n in (1, 2):
            off = (c.want(n) != want)[want != 0]
            assert off.mean() > (0.98 if n == 1 else 0.9)
    for side in ("Y", "dX"):
        c = Small(M, r, side)
        want = c.want()
        assert _bits(want).shape == want.shape and (c.want(2) == want).all()
        assert (c.want(1) == 0).all() and (want != 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("side", ["a", "b"])
@pytest.mark.parametrize("M,r", SIZES)
def test_gradients_see_all_bits_of_their_sums(M, r, side):
    got = _backward(Exact(M, r, side))[1 if side == "a" else 2]
    want = Exact(M, r, side).want()
    bad = got.double().cpu().numpy() != want
    assert not bad.any(), (np.argwhere(bad)[:4], got.cpu().numpy()[bad][:4], want[bad][:4])


@pytest.mark.gpu
@pytest.mark.parametrize("side", ["Y", "dX"])
@pytest.mark.parametrize("M,r", SIZES)
def test_outputs_see_sixteen_bits_of_their_sums(M, r, side):
    import sparse_rank_linear_amd as srl

    c = Small(M, r, side)
    if side == "Y":
        ad, plan = _adapters(c)
        got = srl.adapters_forward(ad, plan, to_dev(_bits(c.X)), base=to_dev(_bits(c.base)))
    else:
        got = _backward(c)[0]
    assert (ob.bits_to_f64(to_host_bits(got)) == c.want()).all()


def _adapters(c):
    import torch

    import sparse_rank_linear_amd as srl

    ad = srl.SalrAdapters(to_dev(_bits(c.a)), to_dev(_bits(c.b)),
                          ranks=torch.from_numpy(c.ranks.astype(np.int32)).cuda(),
                          scales=torch.from_numpy(c.scales.astype(np.float32)).cuda())
    return ad, srl.adapters_plan(torch.from_numpy(c.ids.astype(np.int32)).cuda(), 2)


def _backward(c):
    import sparse_rank_linear_amd as srl

    ad, plan = _adapters(c)
    return srl.adapters_backward(ad, plan, to_dev(_bits(c.X)), to_dev(_bits(c.dY)), base=to_dev(_bits(c.base)))
