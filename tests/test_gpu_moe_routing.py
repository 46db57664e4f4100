"""Router, dispatch and combine on the GPU, with their gradients, against the
float64 oracle (oracle/routing.py).

Tolerances, derived: u = 2^-24 is fp32's half step, h = 2^-8 bf16's.
 - weights: the exponent l - max has an absolute error of u * 2 * 40 at most
   (|l| < 40 here), expf and the division a few u, the sum of up to 4096
   positive terms (64 a lane, then 6 levels) 70 u: together below 256 u of
   the weight.
 - dlogits: p (up - c), the same errors on p and c: 512 u of p (|up| + sum p
   |dw|), and for bf16 h of the value.
 - combine: k + 1 products and sums, (k + 3) u of the sum of magnitudes, and
   h of the result.  dYs: one product, h of it (and u).
 - dweights: D products summed, (D + 8) u of the sum of magnitudes.
Indexes and copies are exact."""

import numpy as np
import pytest

from oracle import bf16 as ob
from oracle import routing as orr
from tests.gpu_util import say, to_dev, to_host_bits

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
NAN, INF = float("nan"), float("inf")


def _srl():
    import sparse_rank_linear_amd as srl

    return srl


def _bf16(x):
    """Values rounded to bf16, as float64 and as bits."""
    bits = ob.f64_to_bits(np.asarray(x, dtype=np.float64))
    return ob.bits_to_f64(bits), bits


def _logits(T, E, half, seed, mask=0.1):
    """Router logits with ties, -inf entries and rows of -inf only."""
    rng = np.random.default_rng(seed)
    x = np.round(rng.standard_normal((T, E)) * 4, 1)
    x[rng.random((T, E)) < mask] = -INF
    if T > 3:
        x[T // 2] = -INF
        x[T // 3] = 1.5
        x[T - 1, 1:] = -INF
    if half:
        fin = np.isfinite(x)
        x[fin] = _bf16(x[fin])[0]
    else:
        x = x.astype(np.float32).astype(np.float64)
    return x


def _up(x, half=False):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(torch.bfloat16 if half else torch.float32)


# T, E, k: one token and many; E around the powers of two, odd, largest; k = E
ROUTE = [(1, 1, 1), (1, 8, 2), (5, 8, 8), (16, 8, 2), (67, 16, 3), (33, 17, 5), (65, 32, 32), (130, 60, 4), (257, 64, 6),
         (64, 65, 7), (31, 128, 8), (19, 160, 6), (12, 256, 8), (9, 257, 4), (7, 512, 10), (6, 1000, 32), (5, 1500, 2),
         (4, 4096, 8), (4, 4095, 1)]


@pytest.mark.parametrize("T,E,k", ROUTE)
@pytest.mark.parametrize("half", [False, True], ids=["f32", "bf16"])
def test_route(T, E, k, half):
    import torch

    srl = _srl()
    say(f"route T={T} E={E} k={k} half={half}")
    x = _logits(T, E, half, seed=T + E)
    d = _up(x, half)
    for renorm in (False, True):
        want_ids, want = orr.route(x, k, renorm)
        ids = torch.full((T + 2, k), 7, dtype=torch.int32, device="cuda")
        w = torch.full((T + 2, k), 7.0, device="cuda")
        if k % 4 == 0:      # (a view that is still 16-byte aligned)
            iv, wv = ids[1:-1], w[1:-1]
        else:
            iv, wv = torch.empty_like(ids[2:]), torch.empty_like(w[2:])
        got_ids, got = srl.moe_route(d, k, renorm=renorm, ids=iv, weights=wv)
        assert np.array_equal(got_ids.cpu().numpy(), want_ids)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= 256 * U * want).all(), err.max()
        if k % 4 == 0:
            assert (ids[0] == 7).all() and (ids[-1] == 7).all() and (w[0] == 7).all() and (w[-1] == 7).all()


@pytest.mark.parametrize("T,E,k", ROUTE)
@pytest.mark.parametrize("half", [False, True], ids=["f32", "bf16"])
def test_route_backward(T, E, k, half):
    srl = _srl()
    say(f"route_backward T={T} E={E} k={k} half={half}")
    x = _logits(T, E, half, seed=T + E + 1)
    rng = np.random.default_rng(T)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for renorm in (False, True):
        ids, w = orr.route(x, k, renorm)
        ids[0, -1] = -1                                 # a choice that was dropped
        dwd = dw.copy()
        dwd[ids < 0] = NAN                              # never used
        want = orr.route_backward(x, ids, np.where(ids < 0, 0, dw), renorm)
        import torch
        dids = torch.from_numpy(ids).cuda()
        got = srl.moe_route_backward(_up(x, half), dids, _up(dwd), renorm=renorm)
        p = np.zeros((T, E))
        for t in range(T):
            keep = np.isin(np.arange(E), ids[t]) if renorm else np.ones(E, bool)
            v = np.where(keep, x[t], -INF)
            if v.max() > -INF:
                p[t] = np.exp(v - v.max()) / np.exp(v - v.max()).sum()
        up = np.zeros((T, E))
        for t in range(T):
            for e, dd in zip(ids[t], dw[t]):
                if e >= 0:
                    up[t, e] += abs(dd)
        tol = 512 * U * p * (up + (p * up).sum(1, keepdims=True)) + (H * np.abs(want) if half else 0) + 1e-38
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= tol).all(), (err / tol).max()
        # in place
        buf = _up(x, half)
        srl.moe_route_backward(buf, dids, _up(dwd), renorm=renorm, dlogits=buf)
        assert torch.equal(buf, got)


@pytest.mark.parametrize("E,k", [(3, 3), (8, 8), (40, 32), (64, 6), (100, 32), (256, 9), (700, 32), (3000, 8)])
def test_route_backward_any_ids(E, k):
    """Choices of the caller's own: the same expert several times (its
    gradients add up), and ids outside the experts, which take no part."""
    import torch

    srl = _srl()
    rng = np.random.default_rng(E)
    T = 21
    x = rng.standard_normal((T, E)).astype(np.float32).astype(np.float64)
    ids = rng.integers(0, max(2, E // 4), (T, k)).astype(np.int32)
    far = rng.random((T, k)) < 0.2
    ids[far] = rng.choice(np.array([-1, -7, E, E + 5, 2 ** 31 - 1, -2 ** 31]), far.sum()).astype(np.int32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dw[0] = 0.0                                         # (a chosen expert with no gradient is chosen all the same)
    for renorm in (False, True):
        want = orr.route_backward(x, ids, dw, renorm)
        got = srl.moe_route_backward(_up(x), torch.from_numpy(ids).cuda(), _up(dw), renorm=renorm)
        scale = np.abs(dw).sum(1, keepdims=True) * 2
        assert (np.abs(got.double().cpu().numpy() - want) <= 512 * U * scale + 1e-38).all()


def test_route_not_finite():
    """A NaN logit is never chosen and makes full-softmax weights NaN; with
    renorm the others stand; +inf is chosen first, its row's weights NaN."""
    srl = _srl()
    x = np.array([[1.0, NAN, 3.0, 2.0], [0.0, INF, 1.0, 2.0], [NAN] * 4, [0.0, 1.0, 2.0, 3.0]])
    ids, w = srl.moe_route(_up(x), 2, renorm=True)
    assert ids.tolist() == [[2, 3], [1, 3], [-1, -1], [3, 2]]
    w = w.cpu().numpy()
    assert np.allclose(w[0], [1 / (1 + np.exp(-1)), 1 / (1 + np.e)], rtol=1e-6) and (w[2] == 0).all()
    assert np.isnan(w[1]).any()
    ids, w = srl.moe_route(_up(x), 2, renorm=False)
    w = w.cpu().numpy()
    assert ids.tolist() == [[2, 3], [1, 3], [-1, -1], [3, 2]] and np.isnan(w[0]).all() and (w[2] == 0).all()
    assert np.isfinite(w[3]).all()


def _ids(T, k, E, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, k), E - 1, dtype=np.int32)
    if kind == "none":
        return np.full((T, k), -1, dtype=np.int32)
    p = rng.random(E) ** 3 + 1e-3                       # uneven experts; the same one twice a token at times
    ids = rng.choice(E, (T, k), p=p / p.sum()).astype(np.int32)
    if kind == "mixed" and ids.size:
        out = rng.random((T, k)) < 0.15
        ids[out] = rng.choice(np.array([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=np.int64), out.sum()).astype(np.int32)
        ids[T - T // 8:] = -1                           # a padded batch
    return ids


def _want_dispatch(ids, E):
    """orr.dispatch by a stable argsort (quick for many slots)."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    slots = np.argsort(key, kind="stable")
    off = np.searchsorted(key[slots], np.arange(E + 1)).astype(np.int32)
    rows = np.full(flat.size, -1, dtype=np.int32)
    slots = slots[: off[-1]].astype(np.int32)
    rows[slots] = np.arange(off[-1])
    return off, rows.reshape(ids.shape), slots


# T, k, E: no token, one, around the sizes where the work is cut, many experts
DISPATCH = [(0, 2, 8), (1, 1, 1), (1, 2, 8), (1, 32, 64), (16, 2, 8), (16, 6, 64), (63, 1, 3), (64, 1, 64), (65, 1, 2),
            (341, 3, 5), (512, 2, 8), (683, 3, 60), (2047, 8, 3), (2731, 6, 2), (8192, 2, 1), (5462, 3, 33), (1024, 1, 4096), (1025, 1, 1024), (2047, 2, 1025), (2049, 2, 8),
            (4099, 6, 64), (11000, 6, 64), (16384, 8, 256), (70001, 1, 2), (33000, 3, 4096),
            (8192, 8, 64), (8192, 8, 65), (40000, 2, 1000)]


@pytest.mark.parametrize("T,k,E", DISPATCH)
@pytest.mark.parametrize("kind", ["mixed", "one", "none"])
def test_dispatch_sort(T, k, E, kind):
    import torch

    srl = _srl()
    say(f"dispatch T={T} k={k} E={E} {kind}")
    ids = _ids(T, k, E, T + E, kind)
    off, rows, slots = _want_dispatch(ids, E)
    if T * k <= 2000:
        o, r, s = orr.dispatch(ids, E)
        assert np.array_equal(o, off) and np.array_equal(r, rows) and np.array_equal(s, slots)
    D = 16
    X, xb = _bf16(np.random.default_rng(T).standard_normal((T, D)))
    n = T * k
    gslots = torch.full((n + 8,), -77, dtype=torch.int32, device="cuda")
    Xs = torch.full((n + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.randint(0, 255, (srl.moe_dispatch_ws_bytes(T, k, E),), dtype=torch.uint8, device="cuda")
    for _ in range(2):                                   # (a workspace with anything in it, then used)
        x2, goff, grows, _ = srl.moe_dispatch(torch.from_numpy(ids).cuda(), E, to_dev(xb), Xs=Xs[:n], slots=gslots[:n],
                                              ws=ws)
        assert np.array_equal(goff.cpu().numpy(), off)
        assert np.array_equal(grows.cpu().numpy(), rows)
        gs = gslots.cpu().numpy()
        assert np.array_equal(gs[: off[-1]], slots) and (gs[off[-1]:] == -77).all()
        got = to_host_bits(Xs)
        assert np.array_equal(got[: off[-1]], xb[slots // k])
        assert (got[off[-1]:] == 0x40E0).all()           # rows behind the last stay (7.0)
    # the sort alone, and without slots
    _, soff, srows, sslots = srl.moe_dispatch(torch.from_numpy(ids).cuda(), E)
    assert torch.equal(soff, goff) and torch.equal(srows, grows)
    assert np.array_equal(sslots.cpu().numpy()[: off[-1]], slots)
    d, o2, r2 = torch.from_numpy(ids).cuda(), torch.empty_like(goff), torch.empty_like(grows)
    assert srl.lib().salr_moe_dispatch(d.data_ptr() or None, T, k, E, None, 0, o2.data_ptr(), r2.data_ptr() or None,
                                       None, None, ws.data_ptr(), ws.numel(),
                                       torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(o2, goff) and torch.equal(r2, grows)


@pytest.mark.parametrize("D", [1, 2, 3, 4, 8, 36, 40, 1000, 1002, 2044, 2048, 2056, 4099, 8192])
def test_dispatch_and_combine_columns(D):
    """Every width, also odd ones, in few and many tokens."""
    import torch

    srl = _srl()
    for T, k, E in ((1, 2, 8), (5, 6, 64), (700, 3, 5)):
        say(f"columns D={D} T={T} k={k}")
        rng = np.random.default_rng(D + T)
        ids = _ids(T, k, E, D + T)
        off, rows, slots = _want_dispatch(ids, E)
        X, xb = _bf16(rng.standard_normal((T, D)))
        Xs, _, grows, _ = srl.moe_dispatch(torch.from_numpy(ids).cuda(), E, to_dev(xb))
        assert np.array_equal(to_host_bits(Xs)[: off[-1]], xb[slots // k])
        # the way back, with everything that must not be used set to NaN
        Ys, yb = _bf16(rng.standard_normal((T * k, D)))
        yb[off[-1]:] = 0x7FC0
        w = rng.standard_normal((T, k)).astype(np.float32)
        w[rows < 0] = NAN
        B, bb = _bf16(rng.standard_normal((T, D)))
        for weights, base in ((w, None), (w, bb), (None, None), (None, bb)):
            want = orr.combine(Ys, rows, weights, None if base is None else B)
            mag = orr.combine(np.abs(Ys), rows, None if weights is None else np.abs(weights),
                              None if base is None else np.abs(B))
            got = srl.moe_combine(to_dev(yb), grows, None if weights is None else _up(weights),
                                  None if base is None else to_dev(base))
            err = np.abs(ob.bits_to_f64(to_host_bits(got)) - want)
            assert (err <= (k + 3) * U * mag + H * np.abs(want) + 1e-38).all()
        dX = srl.moe_dispatch_backward(to_dev(yb), grows)
        assert torch.equal(dX, srl.moe_combine(to_dev(yb), grows))
        # base may be the output's own buffer
        own = to_dev(bb)
        srl.moe_combine(to_dev(yb), grows, _up(w), base=own, Y=own)
        assert torch.equal(own, srl.moe_combine(to_dev(yb), grows, _up(w), base=to_dev(bb)))
        # gradients
        dY, db = _bf16(rng.standard_normal((T, D)))
        keep = torch.full((T * k, D), 7.0, dtype=torch.bfloat16, device="cuda")
        want_y, want_w = orr.combine_backward(dY, Ys, rows, w)
        gy, gw = srl.moe_combine_backward(to_dev(db), to_dev(yb), grows, _up(w), dYs=keep)
        live = np.arange(T * k) < off[-1]
        g = ob.bits_to_f64(to_host_bits(gy))
        assert (g[~live] == 7.0).all()
        assert (np.abs(g - want_y)[live] <= (H + 2 * U) * np.abs(want_y[live]) + 1e-38).all()
        mag = orr.combine_backward(np.abs(dY), np.abs(Ys), rows)[1]
        err = np.abs(gw.double().cpu().numpy() - want_w)
        assert (err <= (D + 8) * U * mag).all() and (gw.cpu().numpy()[rows < 0] == 0).all()
        # unit weights; over Ys's own buffer
        over = to_dev(yb)
        gy1, gw1 = srl.moe_combine_backward(to_dev(db), over, grows, dYs=over)
        assert torch.equal(gw1, gw)
        assert np.array_equal(to_host_bits(gy1)[live], db[slots // k])


@pytest.mark.parametrize("T,k,D", [(70000, 4, 128), (140000, 2, 127), (9000, 1, 4096), (5000, 8, 1024), (3000, 12, 1000),
                                   (70000, 2, 256)])
def test_rows_of_many_megabytes(T, k, D):
    """Gathered rows of 64 MB and more (read past the caches), against the
    same sums in float64 on the device."""
    import torch

    srl = _srl()
    say(f"many megabytes T={T} k={k} D={D}")
    E = 7
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.from_numpy(_ids(T, k, E, T)).cuda()
    half = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    X, base, Ys = half(T, D), half(T, D), half(T * k, D)
    assert Ys.numel() * 2 >= 64 << 20
    w = torch.rand(T, k, generator=g, device="cuda")
    Xs, off, rows, slots = srl.moe_dispatch(ids, E, X)
    n = int(off[-1])
    assert torch.equal(Xs[:n], X[slots[:n].long() // k])
    Ys[n:] = NAN
    w[rows < 0] = NAN
    at = rows.clamp(min=0).long()
    Y, dY = srl.moe_combine(Ys, rows, w, base=base), X
    dYs, dw = srl.moe_combine_backward(dY, Ys, rows, w)
    want, mag = base.double(), base.double().abs()
    for j in range(k):
        ok = (rows[:, j] >= 0)[:, None]
        y = torch.where(ok, Ys[at[:, j]].double(), 0.0)
        part = torch.where(ok, w[:, j, None].double(), 0.0) * y
        want, mag = want + part, mag + part.abs()
        dot = (dY.double() * y).sum(1)
        tol = (D + 8) * U * (dY.double() * y).abs().sum(1)
        assert ((dw[:, j].double() - dot).abs() <= tol).all()
        d = torch.where(ok, w[:, j, None].double() * dY.double(), 0.0)
        err = torch.where(ok, (dYs[at[:, j]].double() - d).abs(), 0.0)
        assert (err <= (H + 2 * U) * d.abs() + 1e-38).all()
    assert ((Y.double() - want).abs() <= (k + 3) * U * mag + H * want.abs() + 1e-38).all()
    assert torch.count_nonzero(dYs[n:]) == 0


def test_rows_outside_are_skipped():
    """Row entries outside [0, R) of any value add nothing and are not
    written; R = 0 reads nothing."""
    import torch

    srl = _srl()
    rows = torch.tensor([[0, 3], [4, -2 ** 31], [2 ** 31 - 1, 1]], dtype=torch.int32, device="cuda")
    Ys = torch.arange(32, device="cuda").reshape(4, 8).to(torch.bfloat16)
    Y = srl.moe_combine(Ys, rows)
    assert torch.equal(Y, torch.stack([Ys[0] + Ys[3], torch.zeros_like(Ys[0]), Ys[1]]))
    dYs, dw = srl.moe_combine_backward(Y, Ys, rows)
    assert torch.equal(dYs[[0, 3, 1, 2]], torch.stack([Y[0], Y[0], Y[2], torch.zeros_like(Y[0])]))
    assert dw[1].tolist() == [0, 0] and dw[2, 0] == 0
    assert torch.count_nonzero(srl.moe_combine(Ys[:0], rows)) == 0


def test_weights_or_rows_alone():
    """Either gradient alone, through the C ABI, equals the one of both."""
    import torch

    srl = _srl()
    T, k, E, D = 37, 3, 6, 264
    ids = torch.from_numpy(_ids(T, k, E, 3)).cuda()
    _, _, rows, _ = srl.moe_dispatch(ids, E)
    Ys, dY = (torch.randn(s, D, device="cuda").to(torch.bfloat16) for s in (T * k, T))
    w = torch.rand(T, k, device="cuda")
    a, b = srl.moe_combine_backward(dY, Ys, rows, w)
    c, d = torch.zeros_like(a), torch.empty_like(b)
    call = lambda ys, dys, dw: srl.lib().salr_moe_combine_backward(
        dY.data_ptr(), ys, T * k, rows.data_ptr(), w.data_ptr(), T, k, D, dys, dw,
        torch.cuda.current_stream().cuda_stream)
    assert call(None, c.data_ptr(), None) == 0 and call(Ys.data_ptr(), None, d.data_ptr()) == 0
    assert torch.equal(a, c) and torch.equal(b, d)


def test_large_offsets():
    """Row offsets past 2^31 elements in the gathered rows."""
    import torch

    srl = _srl()
    T, k, E, D = 34000, 8, 16, 8192                      # 2.2e9 gathered values
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    X = torch.randn(T, D, generator=g, device="cuda", dtype=torch.bfloat16)
    Xs, off, rows, slots = srl.moe_dispatch(ids, E, X)
    assert int(off[-1]) == T * k
    for s in (0, 1, T * k // 2, T * k - 2, T * k - 1):
        assert torch.equal(Xs[s], X[slots[s] // k])
    w = torch.zeros(T, k, device="cuda")
    w[:, 2] = 1.0
    Y = srl.moe_combine(Xs, rows, w)
    assert torch.equal(Y, X)
    Xs.zero_()
    dYs, dw = srl.moe_combine_backward(X, Xs, rows, w, dYs=Xs)
    assert torch.count_nonzero(dw) == 0
    for t in (0, T // 2, T - 1):
        assert torch.equal(dYs[rows[t, 2]], X[t]) and torch.count_nonzero(dYs[rows[t, 3]]) == 0


def test_results_repeat_and_streams():
    """The same bits on every call, on another stream, and with several
    calls in flight on streams of their own."""
    import torch

    srl = _srl()
    T, k, E, D = 3000, 6, 64, 512
    x = _up(_logits(T, E, False, 5))
    X = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    def chain(stream=None):
        ids, w = srl.moe_route(x, k, stream=stream)
        Xs, off, rows, slots = srl.moe_dispatch(ids, E, X, Xs=None, stream=stream)
        Y = srl.moe_combine(Xs, rows, w, base=X, stream=stream)
        dYs, dw = srl.moe_combine_backward(X, Xs, rows, w, stream=stream)
        dl = srl.moe_route_backward(x, ids, dw, stream=stream)
        n = int(off[-1]) if stream is None else None
        return ids, w, off, rows, Y, dYs, dw, dl
    ref = chain()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [chain(s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for other in got + [chain()]:
        for a, b in zip(ref, other):
            assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a.view(torch.int32),
                               b.view(torch.int16) if b.dtype == torch.bfloat16 else b.view(torch.int32))


def test_captured():
    """Captured into a graph and replayed on new inputs, with eager work
    between the replays, every replay against the eager result."""
    import torch

    srl = _srl()
    for T, k, E, D in ((16, 2, 8, 512), (2500, 6, 64, 256)):
        x, X = torch.empty(T, E, device="cuda"), torch.empty(T, D, device="cuda", dtype=torch.bfloat16)
        x.normal_()
        X.normal_()
        ws = srl.moe_dispatch_workspace(T, k, E)
        def chain():
            ids, w = srl.moe_route(x, k)
            Xs, off, rows, slots = srl.moe_dispatch(ids, E, X, ws=ws)
            Y = srl.moe_combine(Xs, rows, w, base=X)
            dYs, dw = srl.moe_combine_backward(Y, Xs, rows, w)
            return ids, w, off, rows, slots, Xs, Y, dYs, dw, srl.moe_route_backward(x, ids, dw)
        chain()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = chain()
        for r in range(4):
            x.normal_()
            X.normal_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            for a, b in zip(got, chain()):
                assert torch.equal(a, b)
            torch.cuda.synchronize()


def test_binding_refusals():
    import torch

    srl = _srl()
    x = torch.zeros(4, 8, device="cuda")
    i = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    h = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        srl.moe_route(x.half(), 2)
    with pytest.raises(ValueError):
        srl.moe_route(x[:, ::2], 2)
    with pytest.raises(srl.SalrError, match="INVALID_ARG"):
        srl.moe_route(x, 9)
    with pytest.raises(TypeError):
        srl.moe_route_backward(x, i.long(), torch.zeros(4, 2, device="cuda"))
    with pytest.raises(ValueError):
        srl.moe_route_backward(x, i, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(ValueError):
        srl.moe_dispatch(i, 8, h)                        # 8 rows for 4 tokens
    with pytest.raises(ValueError):
        srl.moe_dispatch(i, 8, None, Xs=h)
    with pytest.raises(srl.SalrError, match="WORKSPACE"):
        srl.moe_dispatch(i, 8, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        srl.moe_combine(h.float(), i)
    with pytest.raises(ValueError):
        srl.moe_combine(h, i, torch.zeros(4, 1, device="cuda"))
    with pytest.raises(ValueError, match="on"):
        srl.moe_combine(h, i, torch.zeros(4, 2))
    with pytest.raises(srl.SalrError, match="INVALID_ARG"):
        srl.moe_combine(h[:4], i, Y=h[:4])


@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (100, 4), (256, 32), (700, 8), (4096, 5)])
@pytest.mark.parametrize("half", [False, True], ids=["f32", "bf16"])
def test_route_backward_rows_without_ids(E, k, half):
    """A row none of whose ids is an expert gets zeros, also where its logits
    are NaN or infinite (a dropped token's are whatever was left there); the
    rows beside it are what they are without it."""
    import torch

    srl = _srl()
    rng = np.random.default_rng(E)
    T = 13
    x = _bf16(rng.standard_normal((T, E)))[0]
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dead = [1, 2, 4, 7, 8, 12]
    ids[dead] = rng.choice(np.array([-1, -2 ** 31, E, 2 ** 31 - 1]), (len(dead), k)).astype(np.int32)
    clean = [srl.moe_route_backward(_up(x, half), torch.from_numpy(ids).cuda(), _up(dw), renorm=r)
             for r in (False, True)]
    x[1, 0] = x[2, E - 1] = x[4, E // 2] = NAN
    x[7, 1], x[8, E - 1] = INF, INF
    x[8, 0], x[12] = NAN, NAN
    dw[dead] = NAN
    for renorm in (False, True):
        assert (orr.route_backward(x, ids, np.where(ids < 0, 0, dw), renorm)[dead] == 0).all()
        got = srl.moe_route_backward(_up(x, half), torch.from_numpy(ids).cuda(), _up(dw), renorm=renorm)
        assert torch.count_nonzero(got[dead]) == 0
        alive = [t for t in range(T) if t not in dead]
        assert torch.isfinite(got).all() and torch.equal(got[alive], clean[renorm][alive])


def test_dispatch_workspace_is_as_long_as_it_says():
    """A workspace whose elements share bytes or leave some out is refused."""
    import torch

    srl = _srl()
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    n = srl.moe_dispatch_ws_bytes(4, 2, 8)
    for ws in (torch.zeros(16, dtype=torch.uint8, device="cuda").repeat(1, 1).expand(n, 16),
               torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="ws"):
            srl.moe_dispatch(ids, 8, ws=ws)
    assert srl.moe_dispatch(ids, 8, ws=torch.zeros(n // 4, dtype=torch.int32, device="cuda"))[1].tolist() == [0] + [8] * 8


# Slots around the sizes where another form of the dispatch takes over: 12288
# slots (one launch), 16384 chunk counts (12289 slots in 13 chunks of 1260 or
# 1261 experts), 2^20 slots.
@pytest.mark.parametrize("T,k,E", [(12287, 1, 64), (12288, 1, 64), (12289, 1, 64), (4095, 3, 8), (4096, 3, 8),
                                   (4097, 3, 8), (6143, 2, 2000), (6144, 2, 2000), (6145, 2, 2000), (7001, 1, 300),
                                   (12289, 1, 1260), (12289, 1, 1261), ((1 << 20) - 1, 1, 8), (1 << 20, 1, 8),
                                   ((1 << 20) + 1, 1, 8), (1 << 18, 4, 256), ((1 << 18) + 1, 4, 256),
                                   (174762, 6, 64), (174763, 6, 64), (300000, 8, 1025)])
def test_dispatch_sort_where_forms_change(T, k, E):
    import torch

    srl = _srl()
    say(f"dispatch forms T={T} k={k} E={E}")
    ids = _ids(T, k, E, T + E)
    off, rows, slots = _want_dispatch(ids, E)
    n, D = T * k, 8
    X = torch.randint(-2 ** 15, 2 ** 15, (T, D), device="cuda", dtype=torch.int16).view(torch.bfloat16)
    Xs = torch.full((n + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    gslots = torch.full((n + 8,), -77, dtype=torch.int32, device="cuda")
    d = torch.from_numpy(ids).cuda()
    _, goff, grows, _ = srl.moe_dispatch(d, E, X, Xs=Xs[:n], slots=gslots[:n])
    live = int(off[-1])
    assert np.array_equal(goff.cpu().numpy(), off) and np.array_equal(grows.cpu().numpy(), rows)
    assert np.array_equal(gslots.cpu().numpy()[:live], slots) and (gslots[live:] == -77).all()
    want = X.view(torch.int16)[torch.from_numpy(slots).cuda().long() // k]
    assert torch.equal(Xs.view(torch.int16)[:live], want) and (Xs[live:] == 7.0).all()
    _, soff, srows, sslots = srl.moe_dispatch(d, E)       # the sort alone
    assert torch.equal(soff, goff) and torch.equal(srows, grows)
    assert np.array_equal(sslots.cpu().numpy()[:live], slots)


def _route_many(x, k, renorm):
    """orr.route for many rows: a stable descending sort (ties to the lower)."""
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    vals = np.take_along_axis(x, order, 1)
    ids = np.where(vals > -INF, order, -1).astype(np.int32)
    top = np.where(vals[:, :1] > -INF, vals[:, :1], 0.0)
    e = np.exp(vals - top)
    total = e.sum(1, keepdims=True) if renorm else np.exp(x - top).sum(1, keepdims=True)
    return ids, e / np.where(total > 0, total, 1.0)


@pytest.mark.parametrize("T,E,k", [(16384, 8, 2), (16379, 64, 6), (16384, 256, 8), (4099, 320, 8), (70001, 4, 4)])
@pytest.mark.parametrize("half", [False, True], ids=["f32", "bf16"])
def test_route_many_tokens(T, E, k, half):
    """The router and its gradient over thousands of rows, with ties, masked
    entries and masked rows; the tolerances of test_route and
    test_route_backward."""
    import torch

    srl = _srl()
    say(f"route many T={T} E={E} k={k} half={half}")
    x = _logits(T, E, half, seed=T + E + k)
    d = _up(x, half)
    dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    for renorm in (False, True):
        want_ids, want = _route_many(x, k, renorm)
        few = np.r_[0:40, T // 3, T // 2, T - 1]
        o_ids, o_w = orr.route(x[few], k, renorm)
        assert np.array_equal(o_ids, want_ids[few]) and np.allclose(o_w, want[few], rtol=1e-12, atol=0)
        ids, w = srl.moe_route(d, k, renorm=renorm)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert (np.abs(w.double().cpu().numpy() - want) <= 256 * U * want).all()
        dwd = dw.copy()
        dwd[want_ids < 0] = NAN                             # never used
        got = srl.moe_route_backward(d, ids, _up(dwd), renorm=renorm).double().cpu().numpy()
        chosen, at = want_ids >= 0, np.maximum(want_ids, 0)
        p, up, mag = (np.zeros((T, E)) for _ in range(3))
        rows = np.arange(T)[:, None]
        np.add.at(p, (rows, at), np.where(chosen, want, 0.0))
        if not renorm:
            top = x.max(1, keepdims=True)
            p = np.exp(x - np.where(top > -INF, top, 0.0))
            p /= np.where(top > -INF, p.sum(1, keepdims=True), 1.0)
        np.add.at(up, (rows, at), np.where(chosen, dw, 0.0))
        np.add.at(mag, (rows, at), np.where(chosen, np.abs(dw), 0.0))
        grad = p * (up - (p * up).sum(1, keepdims=True))
        assert np.allclose(orr.route_backward(x[few], want_ids[few], dw[few], renorm), grad[few], rtol=1e-9, atol=1e-15)
        tol = 512 * U * p * (mag + (p * mag).sum(1, keepdims=True)) + (H * np.abs(grad) if half else 0) + 1e-38
        assert (np.abs(got - grad) <= tol).all(), (np.abs(got - grad) / tol).max()


@pytest.mark.parametrize("E,k", [(3, 3), (40, 32), (64, 6), (100, 32), (256, 9), (700, 32), (3000, 8), (4096, 32)])
def test_route_backward_repeated_ids(E, k):
    """Choices drawn from at most 2 k experts, so that a row names some of
    them several times, at a tolerance that goes with each probability (as
    test_route_backward's): taking the last of a repeated expert's gradients,
    or leaving out the mean, is far outside it."""
    import torch

    srl = _srl()
    rng = np.random.default_rng(E + k)
    T = 21
    x = rng.standard_normal((T, E)).astype(np.float32).astype(np.float64)
    pool = rng.permutation(E)[: 2 * k]
    ids = pool[rng.integers(0, pool.size, (T, k))].astype(np.int32)
    ids[:, 1] = ids[:, 0]
    ids[rng.random((T, k)) < 0.1] = -1
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for renorm in (False, True):
        want = orr.route_backward(x, ids, dw, renorm)
        last, no_mean, p, mag = (np.zeros((T, E)) for _ in range(4))
        for t in range(T):
            once = {int(e): d for e, d in zip(ids[t], dw[t]) if e >= 0}
            if once:
                last[t] = orr.route_backward(x[t:t + 1], np.array([list(once)]), np.array([list(once.values())]), renorm)
            keep = np.isin(np.arange(E), ids[t]) if renorm else np.ones(E, bool)
            if once:
                v = np.where(keep, x[t], -INF)
                p[t] = np.exp(v - v.max()) / np.exp(v - v.max()).sum()
            for e, d in zip(ids[t], dw[t]):
                if e >= 0:
                    mag[t, e] += abs(d)
                    no_mean[t, e] += p[t, e] * d
        tol = 512 * U * p * (mag + (p * mag).sum(1, keepdims=True)) + 1e-38
        for wrong in (last, no_mean):
            assert (np.abs(wrong - want) > 4 * tol).any()
        got = srl.moe_route_backward(_up(x), torch.from_numpy(ids).cuda(), _up(dw), renorm=renorm)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= tol).all(), (err / tol).max()


def test_route_far_apart():
    """Logits 0 to 200 below the largest: the exponent is off by 2^-24 of the
    distance, so the weights by 256 u as far as floats are normal (2^-126);
    smaller ones may be 0.  A mask of the type's lowest value is a logit like
    others: weight 0 beside finite ones, an even share among themselves."""
    import torch

    srl = _srl()
    gap = np.arange(0, 200, 0.25)
    for half in (False, True):
        x = np.stack([np.full(gap.size, 3.0), 3.0 - gap], 1)
        x = _bf16(x)[0] if half else x
        for renorm in (False, True):
            want_ids, want = orr.route(x, 2, renorm)
            ids, w = srl.moe_route(_up(x, half), 2, renorm=renorm)
            assert np.array_equal(ids.cpu().numpy(), want_ids)
            err = np.abs(w.double().cpu().numpy() - want)
            assert (err <= 256 * U * want + 2.0 ** -126).all()
        low = torch.finfo(torch.bfloat16 if half else torch.float32).min
        ids, w = srl.moe_route(torch.tensor([[low, 1.0, low, 0.0], [low] * 4], device="cuda")
                               .to(torch.bfloat16 if half else torch.float32), 4)
        assert ids.tolist() == [[1, 3, 0, 2], [0, 1, 2, 3]] and w[0, 2:].tolist() == [0, 0] and w[1].tolist() == [0.25] * 4
