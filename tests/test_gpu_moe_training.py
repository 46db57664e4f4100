"""The routing operators, the grouped experts, the adapter backward and the
AdamW step run together, as a layer of experts is served and fine-tuned:

    logits -> moe_route -> moe_dispatch -> moe_forward (up) -> relu^2
    -> moe_forward (down) -> moe_combine (+ the tokens themselves)

backward: moe_combine_backward -> each expert's linear_backward -> the
activation -> linear_backward -> moe_dispatch_backward, and moe_route_backward;
then one adamw_step over every expert's adapters, and a forward that reads
them.  Each value is compared with the float64 layer computed from the
original inputs.

Tolerances: the layers' own (TOL_MAX_REL and TOL_NORMWISE of a product's
output) for each product on the way: two for the outputs, three for the
token gradients and the router's, doubled by relu^2, whose relative error is
twice its input's.  After the step the adapters are bf16: half a step, 2^-8,
on top of the gradient's error through Adam's quotient, which at step 1 is
lr sign(g) wherever the gradient is above its error."""

import numpy as np
import pytest

from oracle import bf16 as ob
from oracle import routing as orr
from oracle import salr as osl
from sparse_rank_linear_amd import synth
from tests.gpu_util import TOL_NORMWISE, say, to_dev, upload_encoded

pytestmark = pytest.mark.gpu


def _encode(E, N, K, r, seed):
    rng = np.random.default_rng(seed)
    out = []
    for e in range(E):
        W = synth.make_w(N, K, seed * 10 + e, scale=0.08)
        A = ob.f64_to_bits(rng.standard_normal((r, K)) * 0.08)
        B = ob.f64_to_bits(rng.standard_normal((N, r)) * 0.08)
        out.append(osl.encode(W, K // 2, 0, [A], [B]))
    return out


class _Layer:
    """E experts of one shape: grouped, one by one, and their transposes."""

    def __init__(self, E, N, K, r, seed):
        import sparse_rank_linear_amd as srl

        self.encs = _encode(E, N, K, r, seed)
        self.K = K
        self.moe = srl.SalrMoE.empty(E, N, K, K // 2, r)
        self.single = []
        for e, en in enumerate(self.encs):
            self.moe.set_expert(e, en.masks, en.values, en.offsets, en.A_cat.T.copy(), en.B_cat.T.copy())
            one = upload_encoded(en, K, 0)
            one.a_cat, one.b_cat = self.moe.expert_adapters(e)      # (one storage for both ways)
            self.single.append(one)
        self.lt = [srl.transpose_layer(s) for s in self.single]
        self.grads = [(srl.workspace(4 * r * K).view(_t().float32)[: r * K].view(r, K),
                       srl.workspace(4 * N * r).view(_t().float32)[: N * r].view(N, r)) for _ in self.encs]

    def dense(self, e):
        """Expert e's matrix [N][K] in float64 with the adapters it has now."""
        a, b = (x.double().cpu().numpy() for x in self.moe.expert_adapters(e))
        return osl.decode_dense(self.encs[e].masks, self.encs[e].values, self.K) + b @ a

    def backward(self, X, dY, off):
        """Each expert's gradients; returns dX by rows."""
        import sparse_rank_linear_amd as srl

        dX = _t().zeros_like(X)
        for e, (one, lt, (dA, dB)) in enumerate(zip(self.single, self.lt, self.grads)):
            s, t = int(off[e]), int(off[e + 1])
            x, dy = X[s:t].contiguous(), dY[s:t].contiguous()
            got, _, _ = srl.linear_backward(one, lt, x, dy, dA=dA, dB=dB, need_dx=t > s)
            if t > s:
                dX[s:t] = got
        return dX


def _t():
    import torch

    return torch


def _forward(up, down, x, X, k):
    import sparse_rank_linear_amd as srl

    ids, w = srl.moe_route(x, k)
    Xs, off, rows, _ = srl.moe_dispatch(ids, up.moe.E, X)
    H = srl.moe_forward(up.moe, Xs, off)
    A = _t().relu(H.float()).square().to(_t().bfloat16)
    Ys = srl.moe_forward(down.moe, A, off)
    return ids, w, Xs, off, rows, H, A, Ys, srl.moe_combine(Ys, rows, w, base=X)


def _reference(up, down, x, X, k, G):
    """Output, token gradient, logit gradient and adapters' gradients of
    loss = sum(G * Y), in float64 with autograd."""
    torch = _t()
    ids, _ = orr.route(x, k, True)
    lx = torch.tensor(x, dtype=torch.float64, requires_grad=True)
    tx = torch.tensor(X, dtype=torch.float64, requires_grad=True)
    leaves, Y = [], tx * 1.0
    dense = []
    for layer in (up, down):
        per = []
        for e in range(layer.moe.E):
            a, b = (torch.tensor(v.double().cpu().numpy(), requires_grad=True) for v in layer.moe.expert_adapters(e))
            base = torch.tensor(osl.decode_dense(layer.encs[e].masks, layer.encs[e].values, layer.K))
            leaves.append((a, b))
            per.append(base + b @ a)
        dense.append(per)
    for t in range(x.shape[0]):
        sel = [int(e) for e in ids[t] if e >= 0]
        if not sel:
            continue
        w = torch.softmax(lx[t][sel], 0)
        for c, e in enumerate(sel):
            h = torch.relu(dense[0][e] @ tx[t]).square()
            Y = Y.index_add(0, torch.tensor([t]), (w[c] * (dense[1][e] @ h))[None])
    (Y * torch.tensor(G)).sum().backward()
    zero = lambda p: (np.zeros(p.shape) if p.grad is None else p.grad.numpy())
    return (Y.detach().numpy(), tx.grad.numpy(), lx.grad.numpy() if lx.grad is not None else np.zeros(x.shape),
            [(zero(a), zero(b)) for a, b in leaves])


def _near(got, want, times):
    """Normwise within `times` of a product's own tolerance."""
    err = np.linalg.norm(got - want)
    return err <= times * TOL_NORMWISE * np.linalg.norm(want) + 1e-30


# tokens, experts, choices, padded tokens
@pytest.mark.parametrize("T,E,k,pad", [(1, 4, 2, 0), (40, 4, 2, 0), (77, 6, 3, 9), (5, 3, 3, 5)])
def test_layer_forward_backward_step(T, E, k, pad):
    torch = _t()
    import sparse_rank_linear_amd as srl

    say(f"moe layer T={T} E={E} k={k} pad={pad}")
    D, F, r = 256, 384, 16
    up, down = _Layer(E, F, D, r, seed=E), _Layer(E, D, F, r, seed=E + 50)
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, E)).astype(np.float32).astype(np.float64)
    x[T - pad:] = -np.inf
    Xb, Gb = (ob.f64_to_bits(rng.standard_normal((T, D))) for _ in range(2))
    X, G = ob.bits_to_f64(Xb), ob.bits_to_f64(Gb)
    xd, Xd, Gd = torch.tensor(x, dtype=torch.float32, device="cuda"), to_dev(Xb), to_dev(Gb)
    wantY, wantX, wantL, wantP = _reference(up, down, np.where(np.isfinite(x), x, -np.inf), X, k, G)

    ids, w, Xs, off, rows, H, A, Ys, Y = _forward(up, down, xd, Xd, k)
    f64 = lambda t: t.double().cpu().numpy()
    assert _near(f64(Y) - X, wantY - X, 4)
    if pad:
        assert torch.equal(Y[T - pad:], Xd[T - pad:])     # a padded token keeps its row

    dYs, dw = srl.moe_combine_backward(Gd, Ys, rows, w)
    n = int(off[-1])
    dA = down.backward(A, dYs, off)
    dH = torch.where(H.float() > 0, 2 * H.float() * dA.float(), torch.zeros((), device="cuda"))
    dH[n:] = 0
    dXs = up.backward(Xs, dH.to(torch.bfloat16), off)
    dX = srl.moe_dispatch_backward(dXs, rows)
    assert _near(f64(dX), wantX - G, 6)                   # (the base's gradient is G itself)
    if pad < T:
        dl = srl.moe_route_backward(xd, ids, dw)
        assert _near(f64(dl)[: T - pad], wantL[: T - pad], 6)
        assert torch.count_nonzero(dl[T - pad:]) == 0
    grads = [g for layer in (up, down) for g in layer.grads]
    for (gA, gB), (wA, wB) in zip(grads, wantP):
        assert _near(f64(gA), wA, 6) and _near(f64(gB), wB, 6)

    # one step over every adapter of both layers at once
    lr = 2.0 ** -6
    params = [p for layer in (up, down) for e in range(E) for p in layer.moe.expert_adapters(e)]
    flat = [g for pair in grads for g in pair]
    before = [p.double() for p in params]
    plan = srl.adamw_plan(params, flat, **srl.adamw_states(params, bits=8, master=True))
    srl.adamw_step(plan, 1, lr, weight_decay=0.0)
    for p, q, g in zip(params, before, flat):
        step = p.double() - q + lr * g.double().sign()
        clear = g.abs() > 1e-4                            # (eps 1e-8 takes 1e-4 of these updates at most)
        assert (step[clear].abs() <= 2.0 ** -8 * p.double()[clear].abs() + 2e-4 * lr).all()
        assert torch.equal(p.double()[g == 0], q[g == 0])
    # the next forward reads them, grouped and alone
    wantY = _reference(up, down, x, X, k, G)[0]
    Y = _forward(up, down, xd, Xd, k)[-1]
    assert _near(f64(Y) - X, wantY - X, 4)


def test_layer_captured():
    """The served layer in a graph, replayed on new logits and tokens with
    eager work in between."""
    torch = _t()
    import sparse_rank_linear_amd as srl

    T, E, k, D, F, r = 16, 8, 2, 256, 384, 16
    up, down = _Layer(E, F, D, r, seed=3), _Layer(E, D, F, r, seed=4)
    x, X = torch.randn(T, E, device="cuda"), torch.randn(T, D, device="cuda").to(torch.bfloat16)
    bufs = dict(ws=srl.moe_dispatch_workspace(T, k, E), w1=srl.moe_workspace(up.moe, T * k),
                w2=srl.moe_workspace(down.moe, T * k))

    def layer():
        ids, w = srl.moe_route(x, k)
        Xs, off, rows, _ = srl.moe_dispatch(ids, E, X, ws=bufs["ws"])
        H = srl.moe_forward(up.moe, Xs, off, ws=bufs["w1"])
        A = torch.relu(H.float()).square().to(torch.bfloat16)
        return srl.moe_combine(srl.moe_forward(down.moe, A, off, ws=bufs["w2"]), rows, w, base=X)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for _ in range(4):
        x.normal_()
        X.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, layer())
        torch.cuda.synchronize()


def test_expert_adapters_are_the_stored_ones():
    import sparse_rank_linear_amd as srl

    layer = _Layer(3, 48, 64, 8, seed=9)
    for e, en in enumerate(layer.encs):
        a, b = layer.moe.expert_adapters(e)
        assert np.array_equal(a.view(_t().int16).cpu().numpy().view(np.uint16), en.A_cat.T)
        assert np.array_equal(b.view(_t().int16).cpu().numpy().view(np.uint16), en.B_cat.T)
        d = layer.moe.expert(e)
        assert a.data_ptr() == d.a_cat and b.data_ptr() == d.b_cat
    with pytest.raises(ValueError):
        layer.moe.expert_adapters(3)
    assert isinstance(layer.moe, srl.SalrMoE)
