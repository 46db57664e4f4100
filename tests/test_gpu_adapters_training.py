"""The adapters of many requests run as they are used, beside the encoded layer
that all of them share: a batch of several requests through the shared
projection and each one's adapter,

    adapters_plan; linear_forward -> adapters_forward (in place)

the gradients of every adapter at once,

    linear_backward -> adapters_backward (added to its dX)

and a muon_step over all of them, whose results the next batch's forward and a
single token's read.  Each value is compared with the float64 layer computed
from the encoding and the adapters as they are.

Tolerances: the layer's own (TOL_NORMWISE of a product's output) for the shared
projection and once more for the adapters on top of it; float gradients by
2^-8, the rounding of the shared projection's bf16 output having no part in
them.  After the step the adapters are bf16, half a step being 2^-8 of them; X
itself is 1e-4 off at most."""

import numpy as np
import pytest

from oracle import adapters as oa
from oracle import bf16 as ob
from oracle import muon as om
from oracle import salr as osl
from sparse_rank_linear_amd import synth
from tests.gpu_util import TOL_NORMWISE, say, to_dev, upload_encoded

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


def _near(got, want, tol):
    return np.linalg.norm(got - want) <= tol * np.linalg.norm(want) + 1e-30


# tokens of each request, and its adapter (-1: none; 2 takes part in no batch)
@pytest.mark.parametrize("lengths,names", [([1], [0]), ([1] * 9, [0, 3, 1, -1, 3, 0, 0, 1, 3]), ([40, 130, 7, 25], [1, 3, -1, 0]),
                                           ([700, 500], [3, 1])])
def test_batches_of_requests(lengths, names):
    import torch

    import sparse_rank_linear_amd as srl

    say("requests", lengths, names)
    count, N, K, r = 4, 384, 256, 24
    rng = np.random.default_rng(sum(lengths))
    W = synth.make_w(N, K, 5, scale=0.08)
    enc = osl.encode(W, K // 2, 0, [ob.f64_to_bits(rng.standard_normal((16, K)) * 0.08)],
                     [ob.f64_to_bits(rng.standard_normal((N, 16)) * 0.08)])
    layer = upload_encoded(enc, K, 0)
    lt = srl.transpose_layer(layer)
    dense = osl.decode_dense(enc.masks, enc.values, K) + ob.bits_to_f64(enc.B_cat).T @ ob.bits_to_f64(enc.A_cat).T
    ranks, scales = np.array([24, 8, 24, 17]), np.array([1.0, 2.0, 1.0, 0.5])
    ad = srl.SalrAdapters.empty(count, N, K, r)
    ad.a.copy_(to_dev(ob.f64_to_bits(rng.standard_normal((count, r, K)) * 0.1)))
    ad.b.copy_(to_dev(ob.f64_to_bits(rng.standard_normal((count, N, r)) * 0.1)))
    ad.ranks = torch.tensor(ranks, dtype=torch.int32, device="cuda")
    ad.scales = torch.tensor(scales, dtype=torch.float32, device="cuda")
    ids = np.repeat(names, lengths)
    M = len(ids)
    xb, yb = (ob.f64_to_bits(rng.standard_normal((M, d))) for d in (K, N))
    X, dY, xd, yd = ob.bits_to_f64(xb), ob.bits_to_f64(yb), to_dev(xb), to_dev(yb)
    f64 = lambda t: t.double().cpu().numpy()
    weights = lambda: (f64(ad.a), f64(ad.b))

    plan = srl.adapters_plan(torch.tensor(ids, dtype=torch.int32, device="cuda"), count)
    ws = srl.adapters_workspace(ad, M, backward=True)

    def forward():
        Y = srl.linear_forward(layer, xd)
        return srl.adapters_forward(ad, plan, xd, base=Y, Y=Y, ws=ws)

    a, b = weights()
    assert _near(f64(forward()), oa.forward(a, b, ids, ranks, scales, X, X @ dense.T), 2 * TOL_NORMWISE)

    dX, _, _ = srl.linear_backward(layer, lt, xd, yd)
    dX, dA, dB = srl.adapters_backward(ad, plan, xd, yd, base=dX, dX=dX, ws=ws)
    wx, wa, wb = oa.backward(a, b, ids, ranks, scales, X, dY, dY @ dense)
    assert _near(f64(dX), wx, 2 * TOL_NORMWISE) and _near(f64(dA), wa, H) and _near(f64(dB), wb, H)
    assert (dA[2] == 0).all() and (dB[2] == 0).all()

    # one step over every adapter; those without gradients stay
    params = [p for q in range(count) for p in (ad.a[q], ad.b[q])]
    grads = [g for q in range(count) for g in (dA[q], dB[q])]
    opt = srl.muon_plan(params, grads, **srl.muon_states(params))
    before, lr = [f64(p) for p in params], 2.0 ** -4
    srl.muon_step(opt, lr)
    for p, p0, g in zip(params, before, grads):
        want, _, _ = om.step(p0, f64(g), np.zeros(p0.shape), lr, lr_scale=max(1.0, p0.shape[0] / p0.shape[1]) ** 0.5)
        scale = lr * max(1.0, p0.shape[0] / p0.shape[1]) ** 0.5
        assert (np.abs(f64(p) - want) <= H * np.abs(want) + scale * 1e-4).all()
    assert torch.equal(ad.a[2], to_dev(ob.f64_to_bits(before[4]))) and (f64(ad.a[0]) != before[0]).any() == (0 in ids)

    # the next batch and a single token read what the step left
    a, b = weights()
    assert _near(f64(forward()), oa.forward(a, b, ids, ranks, scales, X, X @ dense.T), 2 * TOL_NORMWISE)
    one = srl.adapters_plan(torch.tensor([3], dtype=torch.int32, device="cuda"), count)
    y = srl.adapters_forward(ad, one, xd[:1].contiguous(), base=srl.linear_forward(layer, xd[:1].contiguous()))
    assert _near(f64(y), oa.forward(a, b, [3], ranks, scales, X[:1], X[:1] @ dense.T), 2 * TOL_NORMWISE)
