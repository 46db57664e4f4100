"""8-bit AdamW states rounded by chance (a step with a seed), against the
float64 oracle (oracle/adamw.py).

Tolerances, derived: u = 2^-24 is fp32's half step.
 - one step: a code is one of the two around the exact value, which the
   kernel has to within 5 u of the magnitudes summed (m) or of the value
   (sqrt(v)), and the scale and its inverse to a few u: 16 u.
 - shares: N numbers that take hi with chance p have the mean's standard
   deviation gap sqrt(p (1 - p) / N); 6 of those, and gap 8 / N for chances
   too small for a normal tail.
 - many steps: the expected v is the recurrence's, exactly up to fp32 (64 u a
   step, kept for 1 / (1 - beta2) steps).  Its variance: a step adds at most
   G D, with G the distance of the squared codes around v', at most 0.2656 v'
   ((9/8)^2 - 1), and D the distance of v' from the old code's square under
   the new scale, at most (1 - beta2)(g^2 + v) + r v for a scale whose square
   changes by r; and at most G^2 / 4.  _variance adds that up."""

import numpy as np
import pytest

from oracle import adamw as oa
from tests.gpu_util import say
from tests.test_gpu_adamw import HYPER, SIZES, U, _before, _f64, _make

pytestmark = pytest.mark.gpu

VALUES = np.unique(oa.code_values()[np.isfinite(oa.code_values())])


def _srl():
    import sparse_rank_linear_amd as srl

    return srl


def _bits(t):
    import torch

    return t.contiguous().view(torch.uint8)


def _codes(t, scale):
    """(values, each element's scale) of stored codes, in float64."""
    per = np.repeat(_f64(scale), 256)[: t.numel()]
    return oa.code_values()[_bits(t).cpu().numpy()] * per, per


def _between(t, scale, want, err, root):
    got, per = _codes(t, scale)
    live = per > 0
    assert (got[~live] == 0).all()
    got, want, err, per = got[live] / per[live], want[live], err[live], per[live]
    lo, hi = (want - err) / per, (want + err) / per
    if root:
        lo, hi = (np.where(want > 0, np.maximum(x, 2.0 ** -9), x) for x in (lo, hi))
    below = VALUES[np.clip(np.searchsorted(VALUES, lo, side="right") - 1, 0, VALUES.size - 1)]
    above = VALUES[np.clip(np.searchsorted(VALUES, hi, side="left"), 0, VALUES.size - 1)]
    assert ((below <= got) & (got <= above)).all()


@pytest.mark.parametrize("p_half,g_half,master", [(True, False, False), (True, True, False), (True, False, True),
                                                  (True, True, True), (False, False, False), (False, True, False)])
def test_random_codes(p_half, g_half, master):
    """Parameters, masters and scales are those of a step without a seed, bit
    for bit; every code is one of the two around the exact value; the same
    seed and step give the same codes, others others."""
    import torch

    srl = _srl()
    say(f"random codes p_half={p_half} g_half={g_half} master={master}")
    kinds = ("m", "v", "m_scale", "v_scale")
    ends = []
    for seed, t in ((None, 7), (11, 7), (11, 7), (12, 7), (11, 8)):
        params, grads, st = _make(SIZES, p_half, g_half, 8, master, seed=5)
        before = _before(params, grads, st, 8)
        srl.adamw_step(srl.adamw_plan(params, grads, **st), t, 1e-3, seed=seed, **HYPER)
        ends.append((params, st))
    torch.cuda.synchronize()
    (near_p, near), (got_p, got), (_, again), (_, other_seed), (_, other_step) = ends
    for a, b in zip(near_p + near["m_scale"] + near["v_scale"] + (near["master"] or []),
                    got_p + got["m_scale"] + got["v_scale"] + (got["master"] or [])):
        assert torch.equal(_bits(a), _bits(b))
    flat = lambda st, k: torch.cat([_bits(x) for x in st[k]])
    for k in kinds:
        assert torch.equal(flat(got, k), flat(again, k))
        if not k.endswith("scale"):
            for st in (near, other_seed, other_step):
                assert (flat(st, k) != flat(got, k)).float().mean() > 0.1
    for i, (p0, g0, m0, v0) in enumerate(before):
        if p0.size == 0:
            continue
        _, m, v = oa.step(p0, g0, m0, v0, 7, 1e-3, **HYPER)
        size = HYPER["beta1"] * np.abs(m0) + (1 - HYPER["beta1"]) * np.abs(g0)
        _between(got["m"][i], got["m_scale"][i], m, 16 * U * size, False)
        _between(got["v"][i], got["v_scale"][i], np.sqrt(v), 16 * U * np.sqrt(v), True)


def _step_from_zero(g, seed, t=1):
    """Stored (m, s) in float64, [tensor][n], after one step from zero states."""
    import torch

    srl = _srl()
    p = [torch.zeros_like(x) for x in g]
    st = srl.adamw_states(p, bits=8)
    srl.adamw_step(srl.adamw_plan(p, g, **st), t, 1e-3, seed=seed)
    return [np.stack([_codes(a, b)[0] for a, b in zip(st[k], st[k + "_scale"])]) for k in ("m", "v")]


def test_random_shares():
    """60 magnitudes over the codes' whole range, the same in each of 4096
    runs: the means of m and of s^2 are the exact ones; steps, seeds and
    tensors choose independently, and so do m and s."""
    import torch

    runs = 4096
    mags = np.float32(2.0) ** -np.linspace(0.03, 17.3, 60, dtype=np.float32)
    run = np.concatenate([[1.0], mags[np.arange(255) % 60]]).astype(np.float32)
    run[1::2] *= -1
    g = torch.from_numpy(np.tile(run, runs)).cuda()
    say("random shares")
    (m, m2), (s, s2) = _step_from_zero([g, g], 77)
    share, up = {}, {}
    for name, power in (("m", 1), ("s", 2)):
        want = np.abs(run).astype(np.float64) * (1 - HYPER["beta1"] if name == "m" else (1 - HYPER["beta2"]) ** 0.5)
        scale = want[0] / 448
        at = want[1:61] / scale                           # (place 1 + e of a run has magnitude e % 60)
        below = np.clip(np.searchsorted(VALUES, at * (1 + 1e-6), side="right") - 1, 0, VALUES.size - 2)
        lo, hi = VALUES[below] ** power, VALUES[below + 1] ** power
        p = np.clip((at ** power - lo) / (hi - lo), 0, 1)
        got = np.abs((m if name == "m" else s).reshape(runs, 256))
        for i in range(60):
            if at[i] < 2.0 ** -9 * 1.01:
                continue                                  # (s takes at least the smallest code)
            vals, exact = got[:, 1 + i::60] ** power, want[1 + i] ** power
            gap = (hi[i] - lo[i]) * scale ** power
            tol = gap * (6 * (p[i] * (1 - p[i]) / vals.size) ** 0.5 + 8 / vals.size) + 64 * U * exact
            assert abs(vals.mean() - exact) <= tol, (name, i)
        spread = lambda first, x: np.tile(np.concatenate([[first], x[np.arange(255) % 60]]), runs)
        share[name] = spread(0.0, p)
        limit = spread(want[0], VALUES[below] * scale) * (1 + 1e-5)       # (the lower code and a little)
        up[name] = lambda x, limit=limit: np.abs(x) > limit
    mid = (share["m"] > 0.2) & (share["m"] < 0.8)
    def independent(a, b, pa, pb):
        same, want = (a == b).mean(), pa * pb + (1 - pa) * (1 - pb)
        assert abs(same - want.mean()) <= 6 * (want * (1 - want)).mean() ** 0.5 / a.size ** 0.5, (same, want.mean())
    a, p = up["m"](m)[mid], share["m"][mid]
    for other in (m2, _step_from_zero([g], 77, t=2)[0][0], _step_from_zero([g], 78)[0][0]):
        independent(a, up["m"](other)[mid], p, p)         # tensors of a plan, steps, seeds
    independent(a[:-1], a[1:], p[:-1], p[1:])             # neighbours
    independent(a, up["s"](s)[mid], p, share["s"][mid])   # m and s of an element


def _variance(g2, top2, beta2):
    """Bound on the variance of stored v after each step (gradients' squares g2
    [steps]; the run's largest v from those of top2), and v itself."""
    v = var = top = 0.0
    c = 1 - beta2
    for g, gt in zip(g2, top2):
        new = beta2 * v + c * g
        square = beta2 ** 2 * (v * v + var) + 2 * beta2 * c * g * v + (c * g) ** 2      # E v'^2
        r = abs(beta2 + c * gt / top - 1) if top > 0 else np.inf
        add = 0.2656 * (beta2 * (c + r) * (v * v + var) + (beta2 * c * g + c * g * (c + r)) * v + (c * g) ** 2) \
            if r < np.inf else np.inf
        var = beta2 ** 2 * var + min(add, 0.2656 ** 2 / 4 * square)
        v, top = new, beta2 * top + c * gt
    return v, var


@pytest.mark.parametrize("beta2,turn,steps", [(0.99, 300, 900), (0.999, 2000, 5000)])
@pytest.mark.parametrize("half", [False, True], ids=["f32", "bf16"])
def test_random_rounding_follows_the_recurrence(beta2, turn, steps, half):
    """Thousands of steps on gradients of random sign, with elements of every
    run whose gradients turn 20 times smaller or larger on the way: the mean
    of v of each kind is the float64 recurrence's, and a last step moves the
    parameters at least as far as float states do (the mean of 1 / sqrt(v) is
    at least that of the mean v, and the mean of |m| at least |mean m|;
    16384 elements with a spread of their own size: 6 / 128).  A v that
    stays at its codes fails both."""
    import torch

    srl = _srl()
    say(f"recurrence beta2={beta2} steps={steps} half={half}")
    n, kinds = 65536, ((1.0, 1.0), (1.0, 0.0625), (0.0625, 1.0), (0.25, 0.25))
    size = [torch.tensor(kinds, device="cuda")[:, i].repeat(n // 4) for i in (0, 1)]
    gen = torch.Generator(device="cuda").manual_seed(21)
    dt = torch.bfloat16 if half else torch.float32
    p = [[torch.zeros(n, device="cuda", dtype=dt)] for _ in range(2)]
    g = [torch.zeros(n, device="cuda", dtype=dt)]
    st = [srl.adamw_states(p[0], bits=8), srl.adamw_states(p[1], bits=32)]
    plans = [srl.adamw_plan(a, g, **s) for a, s in zip(p, st)]
    hyper = dict(beta1=0.9, beta2=beta2, eps=1e-12, weight_decay=0.0)
    for t in range(1, steps + 2):
        sign = torch.randint(0, 2, (n,), generator=gen, device="cuda") * 2 - 1
        g[0].copy_(size[int(t > turn)] * sign)
        for plan, seed in zip(plans, (2024, None)):
            srl.adamw_step(plan, t, 1.0 if t > steps else 0.0, seed=seed, **hyper)
    torch.cuda.synchronize()
    s8 = _codes(st[0]["v"][0], st[0]["v_scale"][0])[0]
    moved = [_f64(a[0]) for a in p]
    top2 = np.ones(steps + 1)                             # (kind 0 keeps each run's largest)
    for i, (a, b) in enumerate(kinds):
        g2 = np.where(np.arange(1, steps + 2) > turn, b, a) ** 2
        v, var = _variance(g2, top2, beta2)
        got = (s8[i::4] ** 2).mean()
        tol = 6 * (var / (n // 4)) ** 0.5 + 64 * U / (1 - beta2) * v
        say(f"  kind {i}: v {got / v:.4f} of the recurrence's, tolerance {tol / v:.4f}")
        assert tol < 0.25 * v and abs(got - v) <= tol
        far = [np.abs(x[i::4]).mean() for x in moved]
        say(f"          moved {far[0] / far[1]:.4f} of float states'")
        assert far[0] >= (1 - 6 / 128) * far[1]


def test_random_rounding_captured():
    """A captured step with a seed, its step number on the device too,
    replayed with eager work between, equals eager steps bit for bit; and the
    states are those of steps whose number the host gives."""
    import torch

    srl = _srl()
    runs = {}
    for how in ("host", "eager", "captured"):
        params, grads, st = _make([3000, 513], True, False, 8, True, seed=9, fresh=True)
        plan = srl.adamw_plan(params, grads, **st)
        dyn, graph = torch.zeros(5, device="cuda"), None
        for t in range(1, 6):
            lr = 1e-3 / t
            dyn.copy_(torch.tensor(srl.adamw_dyn(t, lr, grad_scale=0.5, seeded=True)))
            torch.cuda.synchronize()
            if how == "captured" and graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    srl.adamw_step(plan, 0, 0.0, dyn=dyn, seed=3)
            if how == "captured":
                graph.replay()
            elif how == "eager":
                srl.adamw_step(plan, 0, 0.0, dyn=dyn, seed=3)
            else:
                srl.adamw_step(plan, t, lr, grad_scale=0.5, seed=3)
            torch.cuda.synchronize()
            for g in grads:
                g.mul_(0.9)
        runs[how] = st["m"] + st["v"] + st["m_scale"] + st["v_scale"] + params + st["master"]
    for a, b in zip(runs["eager"], runs["captured"]):
        assert torch.equal(_bits(a), _bits(b))
    for a, b in list(zip(runs["eager"], runs["host"]))[:8]:
        assert torch.equal(_bits(a), _bits(b))


def test_random_rounding_not_finite_and_float_states():
    """NaN, infinite and tiny gradients as without a seed; float states do not
    know the seed; on a stream of its own the same bits."""
    import torch

    srl = _srl()
    p, g = [torch.zeros(600, device="cuda")], [torch.ones(600, device="cuda")]
    g[0][3], g[0][300] = float("nan"), float("inf")
    st = srl.adamw_states(p, bits=8)
    plan = srl.adamw_plan(p, g, **st)
    srl.adamw_step(plan, 1, 1.0, weight_decay=0.0, seed=1)
    first = torch.isfinite(p[0])
    assert not first[3] and not first[300] and first.sum() == 598
    g[0].fill_(1.0)
    srl.adamw_step(plan, 2, 1.0, weight_decay=0.0, seed=1)
    assert (~torch.isfinite(p[0])).nonzero().reshape(-1).tolist() == [3] + list(range(256, 512))
    p, g = [torch.zeros(300, device="cuda")], [torch.full((300,), 1e-37, device="cuda")]
    st = srl.adamw_states(p, bits=8)
    srl.adamw_step(srl.adamw_plan(p, g, **st), 1, 1.0, seed=1)
    assert torch.isfinite(p[0]).all() and torch.count_nonzero(_bits(st["m"][0])) == 0
    for bits, seeds in ((32, (None, 5)), (8, (5, 5))):
        ends = []
        for seed, stream in zip(seeds, (None, torch.cuda.Stream())):
            params, grads, st = _make([70000, 9], False, False, bits, False, seed=4)
            plan = srl.adamw_plan(params, grads, **st)
            torch.cuda.synchronize()
            srl.adamw_step(plan, 3, 1e-3, seed=seed, stream=stream)
            torch.cuda.synchronize()
            ends.append(params + st["m"] + st["v"])
        for a, b in zip(*ends):
            assert torch.equal(_bits(a), _bits(b))


def test_random_rounding_large_tensor():
    """Past 2^32 elements of a tensor the chances are others than at its
    start, and every element is reached."""
    import torch

    srl = _srl()
    n = (1 << 32) + 4099
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 0.3, dtype=torch.bfloat16, device="cuda")
    g[::256] = 1.0
    st = srl.adamw_states([p], bits=8)
    srl.adamw_step(srl.adamw_plan([p], [g], **st), 1, 0.5, weight_decay=0.0, seed=1)
    a, b = (_bits(st["m"][0][i:i + 4096]) for i in (0, 1 << 32))
    assert (a != 0).all() and (b != 0).all() and (a != b).float().mean() > 0.1
    assert torch.equal(_bits(st["m_scale"][0][:16]), _bits(st["m_scale"][0][1 << 24:(1 << 24) + 16]))
    assert p[-1] != 0 and (_bits(st["v"][0][-3:]) != 0).all()


def test_random_rounding_refusals():
    import torch

    srl = _srl()
    p, g = [torch.zeros(64, device="cuda")], [torch.zeros(64, device="cuda")]
    plan = srl.adamw_plan(p, g, **srl.adamw_states(p, bits=8))
    with pytest.raises(ValueError, match="seed"):
        srl.adamw_step(plan, 1, 1e-3, seed=1 << 32)
    with pytest.raises(ValueError, match="dyn"):
        srl.adamw_step(plan, 1, 1e-3, dyn=torch.zeros(4, device="cuda"), seed=1)
    with pytest.raises(ValueError, match="dyn"):
        srl.adamw_step(plan, 1, 1e-3, dyn=torch.zeros(5, device="cuda"))
