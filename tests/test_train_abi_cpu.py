"""Refusals and sizes of the routing and AdamW entry points.  Validation runs
on the host before any device work, so these calls are safe without a GPU."""

import ctypes as C

import pytest
import torch

import sparse_rank_linear_amd as srl
from sparse_rank_linear_amd import binding as B

P = 0x10000000       # a made-up, aligned device address


def _route(logits=P, type=1, T=4, E=8, k=2, renorm=1, ids=P + 4096, weights=P + 8192):
    return srl.lib().salr_moe_route(logits, type, T, E, k, renorm, ids, weights, None)


def test_route_refusals():
    assert _route(T=0) == 0 and _route(T=0, logits=None) == 0
    for bad in (dict(logits=None), dict(ids=None), dict(weights=None), dict(logits=P + 4), dict(ids=P + 8),
                dict(weights=P + 2), dict(type=2), dict(type=-1), dict(T=-1), dict(E=0), dict(E=4097), dict(k=0),
                dict(k=9), dict(E=64, k=33), dict(T=1 << 31), dict(T=(1 << 31) // 2, k=2)):
        assert _route(**bad) == -1, bad
    # what is written overlaps nothing (logits 4 x 8 floats, ids and weights 4 x 2 words)
    for bad in (dict(ids=P + 112), dict(weights=P), dict(weights=P + 4096 + 16), dict(ids=P - 16)):
        assert _route(**bad) == -1, bad
    lib = srl.lib()
    args = [P, 1, 4, 8, 2, 1, P + 4096, P + 8192, P + 16384, None]
    for over in (P + 4096, P + 8192 + 16, P + 16, P - 112):
        assert lib.salr_moe_route_backward(*args[:8], over, None) == -1
    for i in (0, 6, 7, 8):
        for v in (None, P + 4):
            assert lib.salr_moe_route_backward(*args[:i], v, *args[i + 1:]) == -1
    assert lib.salr_moe_route_backward(P, 3, 4, 8, 2, 1, P, P, P, None) == -1
    assert lib.salr_moe_route_backward(None, 0, 0, 8, 2, 1, None, None, None, None) == 0


def _dispatch(ids=P, T=4, k=2, E=8, X=P + 4096, D=64, off=P + 8192, rows=P + 12288, slots=P + 16384, Xs=P + 20480,
              ws=P + 65536, ws_bytes=1 << 20):
    return srl.lib().salr_moe_dispatch(ids, T, k, E, X, D, off, rows, slots, Xs, ws, ws_bytes, None)


def test_dispatch_refusals_and_sizes():
    for bad in (dict(ids=None), dict(rows=None), dict(off=None), dict(X=None), dict(Xs=None), dict(Xs=P + 4096),
                dict(X=P + 4104), dict(slots=P + 4), dict(off=P + 4), dict(D=0), dict(D=(1 << 20) + 1), dict(T=-1),
                dict(k=0), dict(k=33), dict(E=0), dict(E=4097), dict(T=1 << 31), dict(T=0, off=None),
                dict(rows=P + 16), dict(slots=P + 12288), dict(off=P), dict(Xs=P + 4096 + 496), dict(Xs=P - 16),
                dict(ws=P + 12288), dict(slots=P)):
        assert _dispatch(**bad) == -1, bad
    for bad in (dict(ws=None), dict(ws=P + 65544), dict(ws_bytes=16), dict(T=0, ws_bytes=0)):
        assert _dispatch(**bad) == -3, bad
    out = C.c_size_t()
    size = srl.lib().salr_moe_dispatch_ws_bytes
    for args in ((-1, 2, 8), (4, 0, 8), (4, 33, 8), (4, 2, 0), (4, 2, 4097), (1 << 31, 1, 8)):
        assert size(*args, C.byref(out)) == -1
    assert size(4, 2, 8, None) == -1
    # a workspace for T_max serves every smaller T
    for k, E in ((1, 8), (6, 64), (8, 4096)):
        sizes = [srl.moe_dispatch_ws_bytes(T, k, E) for T in range(0, 200000, 997)]
        assert sizes == sorted(sizes) and sizes[0] >= E * 4 and sizes[-1] <= 64 * E * 4 + 256


def test_combine_refusals():
    lib = srl.lib()
    good = dict(Ys=P, R=8, rows=P + 4096, weights=P + 8192, base=P + 12288, T=4, k=2, D=64, Y=P + 16384)
    call = lambda **kw: lib.salr_moe_combine(*{**good, **kw}.values(), None)
    assert call(T=0) == 0
    for bad in (dict(Ys=None), dict(rows=None), dict(Y=None), dict(Y=P), dict(Ys=P + 2), dict(rows=P + 4),
                dict(weights=P + 4), dict(base=P + 8), dict(Y=P + 16386), dict(Y=P + 1008), dict(Y=P + 4096 - 16),
                dict(Y=P + 8192), dict(base=P + 16384 + 16), dict(R=-1), dict(T=-1), dict(k=0),
                dict(k=33), dict(D=0), dict(D=(1 << 20) + 1), dict(R=1 << 31)):
        assert call(**bad) == -1, bad
    good = dict(dY=P, Ys=P + 65536, R=8, rows=P + 4096, weights=P + 8192, T=4, k=2, D=64, dYs=P + 16384,
                dweights=P + 32768)
    back = lambda **kw: lib.salr_moe_combine_backward(*{**good, **kw}.values(), None)
    assert back(T=0) == 0 and back(dYs=None, dweights=None) == 0
    for bad in (dict(dY=None), dict(Ys=None), dict(rows=None), dict(dYs=P), dict(dY=P + 2), dict(dYs=P + 2),
                dict(dweights=P + 4), dict(weights=P + 4), dict(dYs=P + 496), dict(dYs=P + 65536 + 128),
                dict(dweights=P + 65536 + 1008), dict(dweights=P + 8192), dict(dweights=P + 16384), dict(R=-1), dict(T=-1), dict(k=0), dict(k=33), dict(D=0)):
        assert back(**bad) == -1, bad


def _tensor(i, n=1000, **kw):
    base = P + i * 0x100000
    t = B.salr_adamw_tensor_t(base, base + 0x10000, base + 0x20000, base + 0x30000, None, None, None, n)
    for key, v in kw.items():
        setattr(t, key, v)
    return t


def _plan(tensors, p=0, g=1, s=0, table=P, nbytes=1 << 20, count=None, out=True):
    arr = (B.salr_adamw_tensor_t * max(len(tensors), 1))(*tensors)
    d = B.salr_adamw_plan_t()
    return srl.lib().salr_adamw_plan(arr, len(tensors) if count is None else count, p, g, s, table, nbytes,
                                     C.byref(d) if out else None, None)


def test_adamw_plan_refusals():
    a, b = _tensor(1), _tensor(2)
    assert _plan([a, b], nbytes=64) == -3 and _plan([a, b], table=None) == -3 and _plan([a, b], table=P + 8) == -3
    assert _plan([a], out=False) == -1 and _plan([a], count=-1) == -1
    assert srl.lib().salr_adamw_plan(None, 1, 0, 1, 0, P, 1 << 20, C.byref(B.salr_adamw_plan_t()), None) == -1
    for kw in (dict(p=2), dict(g=-1), dict(s=2)):
        assert _plan([a], **kw) == -1
    for field in ("p", "g", "m", "v"):
        assert _plan([_tensor(1, **{field: None})]) == -1
        assert _plan([_tensor(1, **{field: P + 4})]) == -1
    assert _plan([_tensor(1, n=-1)]) == -1 and _plan([_tensor(1, n=1 << 40)]) == -1
    assert _plan([a], s=1) == -1                                        # 8-bit states without scales
    s8 = dict(m_scale=P + 0x40000, v_scale=P + 0x50000)
    assert _plan([_tensor(1, **s8)], s=1, nbytes=0) == -3
    assert _plan([_tensor(1, m_scale=P + 0x40002, v_scale=P + 0x50000)], s=1) == -1
    assert _plan([_tensor(1, m_scale=P + 0x40004, v_scale=P + 0x5000C)], s=1, nbytes=0) == -3
    # masters: all or none, bf16 parameters only
    m1, m2 = _tensor(1, master=P + 0x60000 + 0x100000), _tensor(2, master=P + 0x60000 + 0x200000)
    assert _plan([m1, m2], nbytes=0) == -3 and _plan([m1, b]) == -1 and _plan([b, m1]) == -1
    assert _plan([m1, m2], p=1) == -1
    # what a step writes is disjoint, and gradients are not written
    assert _plan([a, a]) == -1
    assert _plan([a, _tensor(2, p=a.p + 1024)]) == -1
    assert _plan([a, _tensor(2, m=a.v)]) == -1 and _plan([_tensor(1, m=a.v)]) == -1
    assert _plan([a, _tensor(2, g=a.m)]) == -1 and _plan([_tensor(1, g=a.p)]) == -1
    assert _plan([a, _tensor(2, g=a.g)], nbytes=0) == -3                # one gradient for two tensors is fine
    assert _plan([a, _tensor(2, n=0, p=None, g=None, m=None, v=None)], nbytes=0) == -3
    out = C.c_size_t()
    size = srl.lib().salr_adamw_plan_bytes
    n = (C.c_int64 * 2)(5, 1 << 40)
    assert size(n, 2, C.byref(out)) == -1 and size(n, 1, C.byref(out)) == 0 and size(None, 1, C.byref(out)) == -1
    assert size(n, -1, C.byref(out)) == -1 and size(n, 1, None) == -1
    n[1] = 2048 << 24
    assert size(n, 2, C.byref(out)) == -1                               # more runs than one launch has


def test_adamw_step_refusals():
    lib = srl.lib()
    d = B.salr_adamw_plan_t(P, 0, 1, 0, 1, 0, 0)
    args = lambda **kw: B.salr_adamw_step_args_t(*{**dict(step=1, lr=1e-3, b1=.9, b2=.999, eps=1e-8, wd=.01, gs=1.),
                                                   **kw}.values())
    run = lambda a, dyn=None, d=d: lib.salr_adamw_step(C.byref(d), C.byref(a), dyn, None)
    assert run(args()) == 0                                             # (no chunks: nothing to launch)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(step=0), dict(lr=-1.), dict(lr=nan), dict(b1=1.), dict(b1=-.1), dict(b2=1.), dict(b2=nan),
                dict(eps=-1.), dict(eps=nan), dict(wd=-1.), dict(wd=inf)):
        assert run(args(**bad)) == -1, bad
    assert run(args(step=0, lr=-1.), dyn=P) == 0 and run(args(), dyn=P + 2) == -1
    assert lib.salr_adamw_step(None, C.byref(args()), None, None) == -1
    assert lib.salr_adamw_step(C.byref(d), None, None, None) == -1
    for bad in ((None, 0, 1, 0, 1, 0, 0), (P + 8, 0, 1, 0, 1, 0, 0), (P, -1, 1, 0, 1, 0, 0), (P, 0, -1, 0, 1, 0, 0),
                (P, 0, 1, 2, 1, 0, 0), (P, 0, 1, 0, 7, 0, 0), (P, 0, 1, 0, 1, 2, 0), (P, 0, 1, 1, 1, 0, 1)):
        assert run(args(), d=B.salr_adamw_plan_t(*bad)) == -1, bad


def test_binding_refuses_host_tensors():
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    h = torch.zeros(8, 16, dtype=torch.bfloat16)
    for call in (lambda: srl.moe_route(x, 2), lambda: srl.moe_route_backward(x, i, torch.zeros(4, 2)),
                 lambda: srl.moe_dispatch(i, 8), lambda: srl.moe_combine(h, i), lambda: srl.moe_dispatch_backward(h, i),
                 lambda: srl.moe_combine_backward(h[:4], h, i),
                 lambda: srl.adamw_plan([h], [torch.zeros(8, 16)], **srl.adamw_states([h]))):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(ValueError):
        srl.adamw_plan([], [], [], [])
    with pytest.raises(ValueError):
        srl.adamw_plan([h], [], [h], [h])
    with pytest.raises(ValueError):
        srl.adamw_states([h], bits=4)
    st = srl.adamw_states([h, h], bits=8, master=True)
    assert st["m"][0].dtype == torch.float8_e4m3fn and st["m_scale"][1].numel() == 1 and len(st["master"]) == 2
    with pytest.raises(ValueError, match="scale"):
        srl.adamw_plan([h], [h], [h.float()], [h.float()], m_scale=[h.float()], v_scale=[h.float()])


def test_adamw_step_random_refusals():
    lib = srl.lib()
    d = B.salr_adamw_plan_t(P, 0, 1, 0, 1, 1, 0)
    args = lambda **kw: B.salr_adamw_step_args_t(*{**dict(step=1, lr=1e-3, b1=.9, b2=.999, eps=1e-8, wd=.01, gs=1.),
                                                   **kw}.values())
    run = lambda a, dyn=None, seed=5: lib.salr_adamw_step_random(C.byref(d), C.byref(a), seed, dyn, None)
    assert run(args()) == 0 and run(args(), dyn=P) == 0 and run(args(), seed=2 ** 32 - 1) == 0
    for bad in (dict(step=0), dict(lr=-1.), dict(b1=1.), dict(b2=1.), dict(eps=-1.), dict(wd=-1.)):
        assert run(args(**bad)) == -1, bad
    assert run(args(), dyn=P + 2) == -1
    assert lib.salr_adamw_step_random(None, C.byref(args()), 5, None, None) == -1
    assert lib.salr_adamw_step_random(C.byref(d), None, 5, None, None) == -1
    assert C.sizeof(B.salr_adamw_step_args_t) == 56         # (as callers of salr_adamw_step were built)
    for seed in (-1, 2 ** 32):
        with pytest.raises(ValueError, match="seed"):
            srl.adamw_step(None, 1, 1e-3, seed=seed)
    assert srl.adamw_dyn(3, 0.5, seeded=True) == srl.adamw_dyn(3, 0.5) + [3.0]


def test_adamw_plans_stay_within_a_launch():
    """Workgroups of 2048 elements have 256 threads, of 4096 elements 512: a
    launch's threads stay below 2^32 in either."""
    count = 1 << 20
    n = (C.c_int64 * count)(*([7 * 4096] * count))
    out, size = C.c_size_t(), srl.lib().salr_adamw_plan_bytes
    assert size(n, count, C.byref(out)) == 0                            # 14 x 2^20 runs of 2048, 7 x 2^20 of 4096
    n = (C.c_int64 * count)(*([7 * 4096 + 1] * count))
    assert size(n, count, C.byref(out)) == -1                           # 15 x 2^20, and 2^23
    n[0] = 7 * 4096
    assert size(n, count, C.byref(out)) == 0                            # 2^23 - 1
    args = B.salr_adamw_step_args_t(1, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0)
    for state, master, chunks in ((0, 1, 1 << 23), (0, 0, 1 << 24), (1, 0, 1 << 24), (1, 1, 1 << 24)):
        d = B.salr_adamw_plan_t(P, chunks, 1, 0, 1, state, master)
        assert srl.lib().salr_adamw_step(C.byref(d), C.byref(args), None, None) == -1
