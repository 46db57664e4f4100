"""Refusals and sizes of the entry points of the adapters of many requests and
of the orthogonalised step.  Validation runs on the host before any device
work, so these calls are safe without a GPU."""

import ctypes as C

import pytest
import torch

import sparse_rank_linear_amd as srl
from sparse_rank_linear_amd import binding as B

P = 0x10000000       # a made-up, aligned device address


def _adapters(**kw):
    d = dict(count=2, r=8, N=16, K=24, a=P, b=P + 0x10000, ranks=P + 0x20000, scales=P + 0x30000)
    d.update(kw)
    return B.salr_adapters_t(*(d[f] for f, _ in B.salr_adapters_t._fields_))


def _plan_desc(buffer=P + 0x40000, M=5, count=2):
    return B.salr_adapters_plan_t(buffer, M, count)


def test_plan_refusals_and_sizes():
    lib, out = srl.lib(), B.salr_adapters_plan_t()
    call = lambda ids=P, M=5, count=2, buf=P + 0x10000, n=1 << 20, o=out: lib.salr_adapters_plan(
        ids, M, count, buf, n, C.byref(o) if o is not None else None, None)
    for bad in (dict(ids=None), dict(ids=P + 4), dict(M=-1), dict(M=1 << 31), dict(count=0),
                dict(count=srl.ADAPTERS_MAX + 1), dict(o=None), dict(buf=P), dict(buf=P - 16)):
        assert call(**bad) == -1, bad
    for bad in (dict(buf=None), dict(buf=P + 0x10008), dict(n=64)):
        assert call(**bad) == -3, bad
    n = C.c_size_t()
    for args in ((-1, 2), (5, 0), (5, 4097), (1 << 31, 2)):
        assert lib.salr_adapters_plan_bytes(*args, C.byref(n)) == -1
    assert lib.salr_adapters_plan_bytes(5, 2, None) == -1
    for count in (1, 7, 64, 4096):
        sizes = [srl.adapters_plan_bytes(M, count) for M in range(0, 200000, 701)]
        assert sizes == sorted(sizes)                  # (a plan's buffer serves shorter batches)
        assert srl.adapters_plan_bytes(1024, count) <= srl.adapters_plan_bytes(1025, count)
        assert all(s >= 4 * M for M, s in zip(range(0, 200000, 701), sizes))
        # chunks become longer from 16384 tokens on, by 64 every 2048
        for M in (1024, 16384, 18432, 18433, 34816, 65536, 1 << 20, (1 << 20) + 2048):
            assert srl.adapters_plan_bytes(M, count) <= srl.adapters_plan_bytes(M + 1, count), (count, M)
    # as many tokens as every launch has room for
    assert srl.adapters_plan_bytes(1 << 27, 4096) > 4 << 27
    assert lib.salr_adapters_plan_bytes((1 << 27) + 1, 1, C.byref(n)) == -1
    assert lib.salr_adapters_ws_bytes(1, 16, 24, 8, (1 << 27) + 1, 0, C.byref(n)) == -1
    assert call(M=(1 << 27) + 1, n=1 << 40) == -1


def _forward(A=None, plan=None, X=P + 0x100000, base=P + 0x200000, Y=P + 0x300000, ws=P + 0x400000, n=1 << 24):
    A, plan = A or _adapters(), plan or _plan_desc()
    return srl.lib().salr_adapters_forward(C.byref(A), C.byref(plan), X, base, Y, ws, n, None)


SHAPES = (dict(count=0), dict(count=4097), dict(r=0), dict(r=4), dict(r=12), dict(r=264), dict(N=0),
          dict(N=(1 << 20) + 1), dict(K=0), dict(K=20), dict(K=(1 << 20) + 8), dict(a=None), dict(b=None),
          dict(a=P + 2), dict(b=P + 0x10002), dict(ranks=P + 0x20004), dict(scales=P + 0x30008))


def test_forward_refusals():
    for bad in SHAPES:
        assert _forward(_adapters(**bad)) == -1, bad
    for bad in (dict(buffer=None), dict(buffer=P + 8), dict(M=-1), dict(count=3)):
        assert _forward(plan=_plan_desc(**bad)) == -1, bad
    assert _forward(plan=_plan_desc(M=0), X=None, Y=None, ws=None) == 0
    # X 5 x 24 x 2 = 240 bytes, Y 160, a and b 768 and 512, the plan's buffer
    for bad in (dict(X=None), dict(Y=None), dict(X=P + 0x100008), dict(Y=P + 0x300002), dict(base=P + 0x200004),
                dict(Y=P + 0x100000 + 224), dict(Y=P + 0x200000 + 16), dict(Y=P + 752), dict(Y=P + 0x40000),
                dict(ws=P + 0x300000 + 144), dict(ws=P + 0x100000), dict(Y=P + 0x20000), dict(Y=P + 0x30000)):
        assert _forward(**bad) == -1, bad
    for bad in (dict(ws=None), dict(ws=P + 0x400008), dict(n=16), dict(Y=P + 0x200000, n=0)):
        assert _forward(**bad) == -3, bad
    assert srl.lib().salr_adapters_forward(None, C.byref(_plan_desc()), P, P, P, P, 0, None) == -1
    assert srl.lib().salr_adapters_forward(C.byref(_adapters()), None, P, P, P, P, 0, None) == -1


def _backward(A=None, plan=None, X=P + 0x100000, dY=P + 0x200000, base=P + 0x300000, dX=P + 0x400000, dA=P + 0x500000,
              dB=P + 0x600000, ws=P + 0x700000, n=1 << 24):
    A, plan = A or _adapters(), plan or _plan_desc()
    return srl.lib().salr_adapters_backward(C.byref(A), C.byref(plan), X, dY, base, dX, dA, dB, ws, n, None)


def test_backward_refusals():
    for bad in SHAPES:
        assert _backward(_adapters(**bad)) == -1, bad
    assert _backward(_adapters(N=20)) == -2
    for bad in (dict(X=None), dict(dY=None), dict(dA=None), dict(dB=None), dict(X=P + 2), dict(dY=P + 0x200004),
                dict(base=P + 0x300008), dict(dX=P + 0x400002), dict(dA=P + 0x500004), dict(dB=P + 0x600008),
                dict(dX=P + 0x100000), dict(dX=P + 0x300000 + 16), dict(dA=P), dict(dB=P + 0x500000 + 1520),
                dict(dB=P + 0x10000), dict(ws=P + 0x600000), dict(dA=P + 0x40000)):
        assert _backward(**bad) == -1, bad
    for bad in (dict(ws=None), dict(n=16), dict(ws=P + 0x700004), dict(dX=P + 0x300000, n=0), dict(dX=None, n=0)):
        assert _backward(**bad) == -3, bad


def test_workspace_sizes():
    out = C.c_size_t()
    size = srl.lib().salr_adapters_ws_bytes
    for args in ((0, 16, 24, 8, 5, 0), (2, 0, 24, 8, 5, 0), (2, 16, 20, 8, 5, 0), (2, 16, 24, 12, 5, 0),
                 (2, 16, 24, 8, -1, 0), (2, 16, 24, 8, 1 << 31, 1)):
        assert size(*args, C.byref(out)) == -1
    assert size(2, 20, 24, 8, 5, 1, C.byref(out)) == -2 and size(2, 20, 24, 8, 5, 0, C.byref(out)) == 0
    assert size(2, 16, 24, 8, 5, 0, None) == -1
    # a workspace for M_max serves every smaller batch
    for backward in (False, True):
        for count, r in ((1, 8), (64, 64), (4096, 256)):
            sizes = [srl.adapters_ws_bytes(count, 4096, 4096, r, M, backward) for M in range(0, 100000, 499)]
            assert sizes == sorted(sizes) and sizes[0] > 0


def _tensor(i, rows=16, cols=40, **kw):
    base = P + i * 0x100000
    t = B.salr_muon_tensor_t(base, base + 0x10000, base + 0x20000, None, rows, cols, 1.0)
    for key, v in kw.items():
        setattr(t, key, v)
    return t


def _muon_plan(tensors, p=1, g=1, table=P, nbytes=1 << 28, count=None, out=True):
    arr = (B.salr_muon_tensor_t * max(len(tensors), 1))(*tensors)
    d = B.salr_muon_plan_t()
    return srl.lib().salr_muon_plan(arr, len(tensors) if count is None else count, p, g, table, nbytes,
                                    C.byref(d) if out else None, None)


def test_muon_plan_refusals():
    a, b = _tensor(1), _tensor(2)
    far = dict(table=0x7000000000)
    assert _muon_plan([a, b], nbytes=64, **far) == -3 and _muon_plan([a, b], table=None) == -3
    assert _muon_plan([a, b], table=far["table"] + 8) == -3
    assert _muon_plan([a], out=False) == -1 and _muon_plan([a], count=-1) == -1
    for kw in (dict(p=2), dict(g=-1)):
        assert _muon_plan([a], **kw, **far) == -1
    for field in ("p", "g", "m"):
        assert _muon_plan([_tensor(1, **{field: None})], **far) == -1
        assert _muon_plan([_tensor(1, **{field: P + 4})], **far) == -1
    for kw in (dict(rows=-1), dict(cols=-1), dict(lr_scale=float("nan"))):
        assert _muon_plan([_tensor(1, **kw)], **far) == -1
    for kw in (dict(rows=257, cols=257), dict(rows=256, cols=1 << 21)):
        assert _muon_plan([_tensor(1, **kw)], **far) == -2
    m1, m2 = _tensor(1, master=P + 0x130000), _tensor(2, master=P + 0x230000)
    assert _muon_plan([m1, m2], p=0, nbytes=0, **far) == -3
    assert _muon_plan([m1, b], p=0, **far) == -1 and _muon_plan([m1, m2], p=1, **far) == -1
    assert _muon_plan([a, a], **far) == -1                                  # written twice
    assert _muon_plan([_tensor(1, g=P + 0x100000 + 16)], **far) == -1        # a gradient that is written
    assert _muon_plan([a], table=P + 0x120000 + 256) == -1                   # the table on the momentum
    assert _muon_plan([_tensor(1, lr_scale=1e39)], **far) == -1
    # empty matrices need nothing
    assert _muon_plan([_tensor(1, p=None, g=None, m=None, rows=0)], nbytes=0, **far) == -3


def test_muon_sizes_and_step_refusals():
    lib, out = srl.lib(), C.c_size_t()
    i64 = lambda *v: (C.c_int64 * len(v))(*v)
    assert lib.salr_muon_plan_bytes(i64(16), i64(40), 1, C.byref(out)) == 0 and out.value > 0
    assert lib.salr_muon_plan_bytes(i64(16), i64(40), 1, None) == -1
    assert lib.salr_muon_plan_bytes(None, i64(40), 1, C.byref(out)) == -1
    assert lib.salr_muon_plan_bytes(i64(-1), i64(40), 1, C.byref(out)) == -1
    assert lib.salr_muon_plan_bytes(i64(300), i64(300), 1, C.byref(out)) == -2
    assert lib.salr_muon_plan_bytes(None, None, 0, C.byref(out)) == 0
    # shorter sides above 112 have launches with room for 65535 matrices; below, they need no more
    for side, n, want in ((113, 65535, 0), (113, 65536, -2), (112, 65536, 0)):
        rows, cols = i64(*[side] * n), i64(*[200] * n)
        assert lib.salr_muon_plan_bytes(rows, cols, n, C.byref(out)) == want
    plan = B.salr_muon_plan_t(P, 1, 1, 1, 0)
    plan.matrices[0], plan.chunks[0] = 1, 1
    args = dict(lr=0.1, momentum=0.9, weight_decay=0.0, eps=1e-7, grad_scale=1.0, a=3.4, b=-4.7, c=2.0, steps=5,
                nesterov=1)
    nan, inf = float("nan"), float("inf")
    step = lambda plan=plan, dyn=None, **kw: lib.salr_muon_step(
        C.byref(plan), C.byref(B.salr_muon_step_args_t(*{**args, **kw}.values())), dyn, None)
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(momentum=1.0), dict(momentum=-0.1), dict(weight_decay=-1.0),
                dict(eps=0.0), dict(eps=inf), dict(grad_scale=nan), dict(a=inf), dict(b=nan), dict(c=inf),
                dict(steps=0), dict(steps=7), dict(dyn=P + 2)):
        assert step(**bad) == -1, bad
    # what no float holds, and an eps beside which squares that underflow would count
    for bad in (dict(lr=1e39), dict(weight_decay=1e39), dict(grad_scale=-1e39), dict(eps=1e-13)):
        assert step(**bad) == -1, bad
    for field, v in (("table", None), ("table", P + 4), ("count", -1), ("p_type", 3), ("g_type", 3), ("has_master", 1),
                     ("count", 0)):
        bad = B.salr_muon_plan_t.from_buffer_copy(plan)
        setattr(bad, field, v)
        assert step(plan=bad) == -1, field
    bad = B.salr_muon_plan_t.from_buffer_copy(plan)
    bad.chunks[3] = -1
    assert step(plan=bad) == -1
    assert lib.salr_muon_step(None, C.byref(B.salr_muon_step_args_t(*args.values())), None, None) == -1
    empty = B.salr_muon_plan_t(P, 0, 1, 1, 0)
    assert step(plan=empty) == 0


def _held(count=4, r=16, K=16, N=16):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    return srl.SalrAdapters(z(count, r, K), z(count, N, r), ranks=torch.full((count,), 5, dtype=torch.int32),
                            scales=torch.ones(count))


def test_descriptor_follows_the_tensors():
    """Another shape, order or type at the same address is seen: the kernels
    write as much as the descriptor says."""
    ad = _held()
    d = ad.descriptor()
    assert (d.count, d.r, d.N, d.K) == (4, 16, 16, 16) and d.a == ad.a.data_ptr() and d.ranks == ad.ranks.data_ptr()
    assert ad.descriptor() is d                                  # (nothing changed)
    for t in ("a", "b", "ranks", "scales"):                      # two of four adapters
        getattr(ad, t).data = getattr(ad, t).data[:2]
    assert ad.descriptor().count == ad.count == 2 and ad.descriptor().a == d.a
    assert srl.adapters_workspace(ad, 5, backward=True).numel() == srl.adapters_ws_bytes(2, 16, 16, 16, 5, True)
    # fewer ranks of as many values: [count][8][32] and [count][32][8] at the same addresses
    ad.a.data, ad.b.data = ad.a.data.view(2, 8, 32), ad.b.data.view(2, 32, 8)
    # (the workspace is sized before anything else has looked at the tensors)
    assert srl.adapters_workspace(ad, 5, backward=True).numel() == srl.adapters_ws_bytes(2, 32, 32, 8, 5, True)
    d = ad.descriptor()
    assert (d.r, d.N, d.K) == (ad.r, ad.N, ad.K) == (8, 32, 32)


@pytest.mark.parametrize("name,change,error", [
    ("a", lambda t: t[:2], ValueError), ("b", lambda t: t[:3], ValueError),
    ("a", lambda t: t.transpose(1, 2), ValueError), ("b", lambda t: t.transpose(1, 2), ValueError),
    ("a", lambda t: t[:, :, ::2], ValueError),
    ("a", lambda t: t.view(dtype=torch.float16), TypeError),
    ("b", lambda t: t.view(dtype=torch.int16), TypeError), ("ranks", lambda t: t[:2], ValueError),
    ("ranks", lambda t: t.view(dtype=torch.float32), TypeError), ("scales", lambda t: t[1:], ValueError),
    ("scales", lambda t: t[::2], ValueError)])
def test_descriptor_refuses_what_no_longer_fits(name, change, error):
    ad = _held()
    ad.descriptor()
    t = getattr(ad, name)
    t.data = change(t.data)
    for _ in range(2):                                           # (each time it is asked)
        with pytest.raises(error):
            ad.descriptor()
        with pytest.raises(error):
            srl.adapters_workspace(ad, 5)


@pytest.mark.parametrize("name", ["a", "b", "c"])
def test_muon_coefficients_are_floats(name):
    """The later steps use them as floats: what no float holds is refused, and
    the largest floats are not."""
    plan = B.salr_muon_plan_t(P, 0, 1, 1, 0)             # (no matrices: nothing is launched)
    args = dict(lr=0.1, momentum=0.9, weight_decay=0.0, eps=1e-7, grad_scale=1.0, a=3.4, b=-4.7, c=2.0, steps=5,
                nesterov=1)
    step = lambda v: srl.lib().salr_muon_step(
        C.byref(plan), C.byref(B.salr_muon_step_args_t(*{**args, name: v}.values())), None, None)
    for v in (1e39, -1e39, 1e308, float("inf"), float("nan")):
        assert step(v) == -1, v
    for v in (3.4e38, -3.4e38, 0.0):
        assert step(v) == 0, v
