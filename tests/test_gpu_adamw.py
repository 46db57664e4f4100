"""The AdamW step on the GPU against the float64 oracle (oracle/adamw.py).

Tolerances, derived: u = 2^-24 is fp32's half step.
 - m, v: constants rounded once (u each), two or three products and a sum:
   5 u of the sum of magnitudes (8-bit states: read back from their codes,
   so their scale adds nothing).
 - p: the quotient has the errors of m (5 u), sqrt(v) (4 u with v's), the
   bias constants, the sum with eps, the division and the product with the
   rate: 24 u of the update's size, where the update's size is taken with
   m's magnitudes; 3 u of |p| for the decay; bf16: 2^-8 of the result.
 - codes: half a step of e4m3, 2^-4 of the value (2^-10 of the scale below
   2^-6 of it), plus 16 u of the value; the scale 8 u of largest / 448."""

import numpy as np
import pytest

from oracle import adamw as oa
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def _srl():
    import sparse_rank_linear_amd as srl

    return srl


def _make(sizes, p_half, g_half, bits, master, seed, fresh=False):
    """Parameters, gradients and states: magnitudes that differ by tensor and
    within it, zeros among the gradients."""
    import torch

    srl = _srl()
    g = torch.Generator(device="cuda").manual_seed(seed)
    norm = lambda n: torch.randn(n, generator=g, device="cuda")
    pt, gt = torch.bfloat16 if p_half else torch.float32, torch.bfloat16 if g_half else torch.float32
    level = lambda i: 10.0 ** (-4 + (i % 5))
    params = [(norm(n) * 0.02).to(pt) for n in sizes]
    grads = [(norm(n) * level(i) * torch.exp(norm(n))).to(gt) for i, n in enumerate(sizes)]
    for t in grads:
        t[::7] = 0
    st = srl.adamw_states(params, bits=bits, master=master)
    if master:
        for m, p in zip(st["master"], params):
            m.add_(norm(m.numel()) * 1e-5)
    if not fresh:
        for i, n in enumerate(sizes):
            m, s = norm(n) * level(i), norm(n).abs() * level(i) * 2
            if bits == 32:
                st["m"][i].copy_(m)
                st["v"][i].copy_(s * s)
            else:                                        # any codes are valid states
                st["m"][i].copy_(torch.randint(0, 127, (n,), generator=g, device="cuda", dtype=torch.uint8)
                                 .view(torch.float8_e4m3fn))
                st["v"][i].copy_(torch.randint(0, 127, (n,), generator=g, device="cuda", dtype=torch.uint8)
                                 .view(torch.float8_e4m3fn))
                st["m_scale"][i].copy_(norm(st["m_scale"][i].numel()).abs() * level(i) / 448)
                st["v_scale"][i].copy_(norm(st["v_scale"][i].numel()).abs() * level(i) / 448)
    return params, grads, st


def _f64(t):
    return t.detach().double().cpu().numpy()


def _states64(st, i, bits):
    """(m, v) of tensor i in float64."""
    import torch

    if bits == 32:
        return _f64(st["m"][i]), _f64(st["v"][i])
    codes = lambda t: t.view(torch.uint8).cpu().numpy()
    return (oa.decode(codes(st["m"][i]), _f64(st["m_scale"][i])),
            oa.decode(codes(st["v"][i]), _f64(st["v_scale"][i])) ** 2)


def _check_codes(t, scale, want, root):
    import torch

    scale, c = _f64(scale), t.view(torch.uint8).cpu().numpy()
    runs = [want[a:a + 256] for a in range(0, want.size, 256)]
    top = np.array([np.abs(r).max() for r in runs])
    live = top >= 2.0 ** -100 * (1 + 1e-6)
    assert (np.abs(scale * 448 - top)[live] <= 8 * U * top[live]).all() and (scale[top < 2.0 ** -100] == 0).all()
    per = np.repeat(scale, 256)[: want.size]
    got = oa.code_values()[c] * per
    tol = np.maximum(np.abs(want) * 2.0 ** -4, per * 2.0 ** -10) + 16 * U * np.abs(want)
    if root:
        tol = np.where((want > 0) & (c == 1), np.maximum(tol, per * 2.0 ** -9), tol)
        assert (c[(want > 0) & (per > 0)] >= 1).all()
    assert (np.abs(got - want) <= tol).all()


def _check_step(before, params, st, t, lr, bits, p_half, hyper=HYPER, gs=1.0):
    for i, (p0, g0, m0, v0) in enumerate(before):
        if p0.size == 0:
            continue
        p, m, v = oa.step(p0, g0, m0, v0, t, lr, grad_scale=gs, **hyper)
        b1, b2 = hyper["beta1"], hyper["beta2"]
        mmag = b1 * np.abs(m0) + (1 - b1) * np.abs(g0 * gs)
        if bits == 32:
            assert (np.abs(_f64(st["m"][i]) - m) <= 5 * U * mmag + 1e-44).all()
            assert (np.abs(_f64(st["v"][i]) - v) <= 6 * U * v + 1e-44).all()
        else:
            _check_codes(st["m"][i], st["m_scale"][i], m, False)
            _check_codes(st["v"][i], st["v_scale"][i], np.sqrt(v), True)
        size = lr * mmag / (1 - b1 ** t) / (np.sqrt(v / (1 - b2 ** t)) + hyper["eps"])
        tol = 24 * U * size + 3 * U * (np.abs(p0) + np.abs(p)) + 1e-44
        if st["master"] is not None:
            assert (np.abs(_f64(st["master"][i]) - p) <= tol).all()
        got = _f64(params[i])
        assert (np.abs(got - p) <= tol * (1 + 2.0 ** -8) + (2.0 ** -8 * np.abs(p) if p_half else 0)).all()


def _before(params, grads, st, bits):
    src = st["master"] if st["master"] is not None else params
    return [(_f64(p), _f64(g), *_states64(st, i, bits)) for i, (p, g) in enumerate(zip(src, grads))]


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 0, 4095, 4096, 4097, 5000, 12345]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_half,g_half,master", [(True, False, False), (True, True, False), (True, False, True),
                                                  (True, True, True), (False, False, False), (False, True, False)])
def test_adamw_steps(bits, p_half, g_half, master):
    """Three steps in a row from set states, every element of every tensor
    checked against one oracle step from the states as they were."""
    import torch

    srl = _srl()
    say(f"adamw bits={bits} p_half={p_half} g_half={g_half} master={master}")
    params, grads, st = _make(SIZES, p_half, g_half, bits, master, seed=bits + p_half)
    plan = srl.adamw_plan(params, grads, **st)
    for t in (1, 2, 50):
        before = _before(params, grads, st, bits)
        srl.adamw_step(plan, t, 1e-3, **HYPER)
        torch.cuda.synchronize()
        _check_step(before, params, st, t, 1e-3, bits, p_half)
        for g in grads:
            g.mul_(-0.5)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_other_settings(bits):
    """From zero states; a gradient scale, betas of 0, a large eps, no decay."""
    srl = _srl()
    for k, (hyper, gs, lr) in enumerate([(dict(beta1=0.0, beta2=0.0, eps=1e-3, weight_decay=0.0), 1.0, 0.1),
                                         (dict(beta1=0.8, beta2=0.9, eps=1.0, weight_decay=0.5), 0.25, 1e-2),
                                         (HYPER, 1e-3, 0.0)]):
        params, grads, st = _make([700, 33], False, False, bits, False, seed=k, fresh=True)
        plan = srl.adamw_plan(params, grads, **st)
        for t in (1, 2):
            before = _before(params, grads, st, bits)
            srl.adamw_step(plan, t, lr, grad_scale=gs, **hyper)
            _check_step(before, params, st, t, lr, bits, False, hyper, gs)


def test_adamw_neighbours_untouched():
    """Tensors inside larger buffers: nothing outside them changes, and a
    plan's tensors are all reached once."""
    import torch

    srl = _srl()
    for bits in (32, 8):
        buf = {}
        n, gap = [9, 2050, 300], 512
        def carve(name, dtype, size):
            base = torch.full((sum(size) + gap * 4 + 64,), 3, dtype=torch.float32, device="cuda").to(dtype)
            buf[name] = (base, [])
            at, out = gap, []
            for s in size:
                out.append(base[at:at + s])
                buf[name][1].append((at, s))
                at = (at + s + 15) // 16 * 16 + gap // 2
            return out
        runs = [-(-s // 256) for s in n]
        code = torch.float8_e4m3fn
        p, m, v = carve("p", torch.bfloat16, n), carve("m", torch.float32 if bits == 32 else code, n), None
        v = carve("v", torch.float32 if bits == 32 else code, n)
        sc = dict(m_scale=carve("ms", torch.float32, runs), v_scale=carve("vs", torch.float32, runs)) if bits == 8 else {}
        g = [torch.ones(s, device="cuda") for s in n]
        srl.adamw_step(srl.adamw_plan(p, g, m, v, **sc), 1, 0.5)
        for name, (base, spans) in buf.items():
            inside = torch.zeros(base.numel(), dtype=torch.bool, device="cuda")
            for a, s in spans:
                inside[a:a + s] = True
            x = base.float()
            assert (x[~inside] == 3).all(), name
            assert (x[inside] != 3).all() if name in ("p", "m", "ms", "vs") or bits == 32 else True, name


def test_adamw_not_finite_and_tiny():
    """A NaN gradient stays in its element; an infinite one in its element,
    or its 8-bit run; values too small for a scale are stored as zeros."""
    import torch

    srl = _srl()
    for bits in (32, 8):
        p, g = [torch.zeros(600, device="cuda")], [torch.ones(600, device="cuda")]
        g[0][3], g[0][300] = float("nan"), float("inf")
        st = srl.adamw_states(p, bits=bits)
        plan = srl.adamw_plan(p, g, **st)
        srl.adamw_step(plan, 1, 1.0, weight_decay=0.0)
        first = torch.isfinite(p[0])
        assert not first[3] and not first[300] and first.sum() == 598
        g[0].fill_(1.0)
        srl.adamw_step(plan, 2, 1.0, weight_decay=0.0)
        bad = (~torch.isfinite(p[0])).nonzero().reshape(-1).tolist()
        assert bad == ([3, 300] if bits == 32 else [3] + list(range(256, 512))), bad
    p, g = [torch.zeros(300, device="cuda")], [torch.full((300,), 1e-37, device="cuda")]
    st = srl.adamw_states(p, bits=8)
    srl.adamw_step(srl.adamw_plan(p, g, **st), 1, 1.0)
    assert torch.isfinite(p[0]).all() and torch.count_nonzero(st["m"][0].view(torch.uint8)) == 0
    assert torch.count_nonzero(st["m_scale"][0]) == 0


def test_adamw8_follows_adamw32():
    """200 steps on a quadratic bowl: the 8-bit run's parameters stay within
    a tenth of the distance travelled of the 32-bit run's (each step's
    direction is off by at most the codes' 2^-4 of m and of its root)."""
    import torch

    srl = _srl()
    n, lr = 4000, 1e-2
    target = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * 4 + 8
    ends = {}
    for bits in (32, 8):
        p, g = [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")]
        plan = srl.adamw_plan(p, g, **srl.adamw_states(p, bits=bits))
        for t in range(1, 201):
            g[0].copy_(p[0] - target)
            srl.adamw_step(plan, t, lr, weight_decay=0.0)
        ends[bits] = p[0].clone()
    far = (ends[32]).abs().mean()
    assert far > 0.5 and (ends[8] - ends[32]).abs().mean() < 0.1 * far


def test_adamw_captured():
    """A captured step with its rate and bias factors on the device, replayed
    with eager work between, equals eager steps bit for bit."""
    import torch

    srl = _srl()
    for bits in (32, 8):
        runs = {}
        for captured in (False, True):
            params, grads, st = _make([3000, 513], True, False, bits, True, seed=9, fresh=True)
            plan = srl.adamw_plan(params, grads, **st)
            dyn = torch.zeros(4, device="cuda")
            graph = None
            for t in range(1, 6):
                lr = 1e-3 / t
                dyn.copy_(torch.tensor(srl.adamw_dyn(t, lr, grad_scale=0.5)))
                torch.cuda.synchronize()
                if captured and graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        srl.adamw_step(plan, 0, 0.0, dyn=dyn)
                if captured:
                    graph.replay()
                else:
                    srl.adamw_step(plan, 0, 0.0, dyn=dyn)
                torch.cuda.synchronize()
                for g in grads:
                    g.mul_(0.9)
            runs[captured] = params + st["m"] + st["v"] + st["master"]
            # the host's arguments give the same up to the rounding of the factors
            if not captured:
                p2, g2, s2 = _make([3000, 513], True, False, bits, True, seed=9, fresh=True)
                plan2 = srl.adamw_plan(p2, g2, **s2)
                srl.adamw_step(plan2, 1, 1e-3, grad_scale=0.5)
                p3, g3, s3 = _make([3000, 513], True, False, bits, True, seed=9, fresh=True)
                plan3 = srl.adamw_plan(p3, g3, **s3)
                dyn.copy_(torch.tensor(srl.adamw_dyn(1, 1e-3, grad_scale=0.5)))
                srl.adamw_step(plan3, 7, 9.0, dyn=dyn)
                for a, b, q in zip(s2["master"], s3["master"], g2):
                    assert ((a - b).abs() <= 16 * U * (a.abs() + 1e-3)).all()
        for a, b in zip(runs[False], runs[True]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_adamw_streams_and_repeat():
    """Steps of different plans on streams of their own; the same bits."""
    import torch

    srl = _srl()
    out = []
    for streams in ([None] * 3, [torch.cuda.Stream() for _ in range(3)]):
        sets = [_make([100000, 77], True, True, 8, False, seed=s) for s in range(3)]
        plans = [srl.adamw_plan(p, g, **st) for p, g, st in sets]
        torch.cuda.synchronize()
        for t in range(1, 4):
            for plan, s in zip(plans, streams):
                srl.adamw_step(plan, t, 1e-2, stream=s)
        torch.cuda.synchronize()
        out.append([x for p, g, st in sets for x in p + st["m"] + st["v"] + st["m_scale"] + st["v_scale"]])
    for a, b in zip(*out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_adamw_large_tensor():
    """A tensor of more than 2^31 elements: its first and last elements."""
    import torch

    srl = _srl()
    n = (1 << 31) + 4099
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[:3], g[-3:], g[n // 2] = 1.0, -2.0, 4.0
    st = srl.adamw_states([p], bits=8)
    srl.adamw_step(srl.adamw_plan([p], [g], **st), 1, 0.5, weight_decay=0.0)
    assert p[:3].tolist() == [-0.5] * 3 and p[-3:].tolist() == [0.5] * 3 and p[n // 2] == -0.5
    assert int(torch.count_nonzero(p[:1 << 20])) == 3 and int(torch.count_nonzero(p[-(1 << 20):])) == 3


def test_adamw_binding_refusals():
    import torch

    srl = _srl()
    p, g = [torch.zeros(64, device="cuda")], [torch.zeros(64, device="cuda")]
    st = srl.adamw_states(p)
    with pytest.raises(ValueError):
        srl.adamw_plan(p, [g[0][:32]], **st)
    with pytest.raises(TypeError):
        srl.adamw_plan(p, [g[0].half()], **st)
    with pytest.raises(TypeError):
        srl.adamw_plan(p + [p[0].bfloat16()], g + g, st["m"] * 2, st["v"] * 2)
    with pytest.raises(ValueError):
        srl.adamw_plan(p, g, [st["m"][0].cpu()], st["v"])
    with pytest.raises(ValueError):
        srl.adamw_plan([torch.zeros(8, 8, device="cuda").t()], g, **st)
    with pytest.raises(srl.SalrError, match="INVALID_ARG"):
        srl.adamw_plan(p * 2, g * 2, st["m"] * 2, st["v"] * 2)           # the same tensor twice
    with pytest.raises(srl.SalrError, match="INVALID_ARG"):
        srl.adamw_plan(p, g, st["m"], st["v"], master=[torch.zeros(64, device="cuda")])   # of a float parameter
    plan = srl.adamw_plan(p, g, **st)
    with pytest.raises(srl.SalrError, match="INVALID_ARG"):
        srl.adamw_step(plan, 0, 1e-3)
    with pytest.raises(ValueError):
        srl.adamw_step(plan, 1, 1e-3, dyn=torch.zeros(3, device="cuda"))
