"""Operators of many adapters at once, for measurement: the adapters of many
requests beside a shared projection with their gradients, and the
orthogonalised step that trains such adapters.

`run` computes them in plain torch (own = False) or through the package
(own = True); `exact` holds the definitions in float64."""

import torch

own = False

# Case keys.  Adapters: M tokens in `requests` runs, one adapter each out of
# `count`; rank r, or with mixed ranks r, r/2, r/4, r/8 in turn; K inputs, N
# outputs; every `bare`-th request has no adapter (0: all have one); plan: the
# pass lays the batch out too (the first of the projections that share it).
# Steps: count pairs of matrices [s][la] and [lb][s], the parameter's and
# gradient's types, a float master copy or none.
MOMENTUM, LR, DECAY, EPS = 0.95, 2e-3, 0.01, 1e-7
STEPS, COEFFICIENTS = 5, (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # the smallest call: one token of one request, rank 16
        {"name": "adapters_token", "op": "forward", "M": 1, "requests": 1, "count": 8, "r": 16, "mixed": False,
         "K": 4096, "N": 4096, "bare": 0, "plan": False},
        # a decode step of 64 requests, each with its own adapter, ranks 64 to 8
        {"name": "adapters_decode", "op": "forward", "M": 64, "requests": 64, "count": 64, "r": 64, "mixed": True,
         "K": 4096, "N": 4096, "bare": 0, "plan": True},
        # a large decode batch over 32 adapters, a feed-forward projection
        {"name": "adapters_decode_wide", "op": "forward", "M": 256, "requests": 256, "count": 32, "r": 16,
         "mixed": False, "K": 4096, "N": 14336, "bare": 0, "plan": False},
        # ragged prompts of 13 requests, some without an adapter
        {"name": "adapters_prefill", "op": "forward", "M": 8191, "requests": 13, "count": 8, "r": 64, "mixed": True,
         "K": 4096, "N": 11008, "bare": 5, "plan": True},
        # a small training batch of four adapters of an expert-sized layer
        {"name": "adapters_grad_small", "op": "backward", "M": 200, "requests": 4, "count": 4, "r": 16,
         "mixed": False, "K": 2048, "N": 1408, "bare": 0, "plan": False},
        # a full training batch, 16 adapters of rank 16
        {"name": "adapters_grad", "op": "backward", "M": 8192, "requests": 32, "count": 16, "r": 16, "mixed": False,
         "K": 4096, "N": 4096, "bare": 0, "plan": True},
        # a ragged one, ranks 80 to 10, some rows without an adapter
        {"name": "adapters_grad_ragged", "op": "backward", "M": 4099, "requests": 9, "count": 6, "r": 80,
         "mixed": True, "K": 4096, "N": 11008, "bare": 4, "plan": False},
        # one 4096 x 4096 layer's adapter pair (rank 80)
        {"name": "step_layer", "op": "step", "count": 1, "s": 80, "la": 4096, "lb": 4096, "p_half": False,
         "g_half": False, "master": False},
        # rank 16 adapters of 64 requests' 4096 x 11008 layer, bf16 gradients
        {"name": "step_requests", "op": "step", "count": 64, "s": 16, "la": 4096, "lb": 11008, "p_half": True,
         "g_half": True, "master": False},
        # three pairs of matrices for each of one layer's 64 experts
        {"name": "step_experts", "op": "step", "count": 192, "s": 80, "la": 2048, "lb": 1408, "p_half": True,
         "g_half": False, "master": False},
        # the feed-forward adapters of 32 blocks (rank 112), float master copies
        {"name": "step_blocks", "op": "step", "count": 64, "s": 112, "la": 4096, "lb": 14336, "p_half": True,
         "g_half": False, "master": True},
        # the widest rank, lengths that are no multiples of anything
        {"name": "step_wide", "op": "step", "count": 3, "s": 253, "la": 8191, "lb": 14337, "p_half": False,
         "g_half": False, "master": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    if rng.random() < 0.45:
        s = _log(rng, 1, 256)
        count = _log(rng, 1, 200)
        la, lb = (_log(rng, s, max(s, min(16384, 20_000_000 // (count * s)))) for _ in range(2))
        p_half = rng.random() < 0.6
        return {"op": "step", "count": count, "s": s, "la": la, "lb": lb, "p_half": p_half,
                "g_half": rng.random() < 0.4, "master": p_half and rng.random() < 0.5}
    op = rng.choice(["forward", "forward", "backward"])
    M = _log(rng, 1, 8192)
    requests = M if M <= 512 and rng.random() < 0.6 else _log(rng, 1, min(M, 64))
    r = rng.choice([8, 16, 16, 24, 32, 64, 80])
    count = _log(rng, 1, max(1, min(64, 512 // r)))
    K, N = (8 * _log(rng, 8, 1400) for _ in range(2))
    return {"op": op, "M": M, "requests": requests, "count": count, "r": r, "mixed": rng.random() < 0.5, "K": K,
            "N": N, "bare": rng.choice([0, 0, 3, 7]), "plan": rng.random() < 0.5}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ranks(case):
    return [max(1, case["r"] >> (a % 4 if case["mixed"] else 0)) for a in range(case["count"])]


def _has_adapter(case, request):
    return not case["bare"] or request % case["bare"] != case["bare"] - 1


def _up8(n):
    return -(-n // 8) * 8


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "step":
        return _prepare_step(case, g)
    M, K, N, r, count, n = (case[k] for k in ("M", "K", "N", "r", "count", "requests"))
    # (each request has one token at least; adapters in an order of the seed's own)
    cuts = torch.sort(torch.randint(0, M - n + 1, (n - 1,), generator=g, device="cuda")).values
    first = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), cuts + torch.arange(1, n, device="cuda")])
    names = torch.randperm(count, generator=g, device="cuda")
    names = names[torch.arange(n, device="cuda") % count]
    live = torch.tensor([_has_adapter(case, i) for i in range(n)], device="cuda")
    names = torch.where(live, names, -1)
    ids = names[torch.searchsorted(first, torch.arange(M, device="cuda"), right=True) - 1].to(torch.int32)
    half = lambda scale, *s: (_normal(g, *s) * scale).to(torch.bfloat16)  # noqa: E731
    st = {"case": case, "ids": ids, "a": half(0.02, count, r, K), "b": half(0.02, count, N, r),
          "ranks": torch.tensor(_ranks(case), dtype=torch.int32, device="cuda"),
          "scales": 0.5 + 1.5 * torch.rand(count, generator=g, device="cuda"), "X": half(1.0, M, K)}
    if case["op"] == "forward":
        st.update(base=half(1.0, M, N), Y=torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
    else:
        st.update(dY=half(1.0, M, N), base=half(1.0, M, K), dX=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"),
                  dA=torch.empty(count, r, K, device="cuda"), dB=torch.empty(count, N, r, device="cuda"))
    if own:
        import sparse_rank_linear_amd as srl
        st["adapters"] = srl.SalrAdapters(st["a"], st["b"], ranks=st["ranks"], scales=st["scales"])
        st["plan"] = srl.adapters_plan(ids, count)
        st["ws"] = srl.adapters_workspace(st["adapters"], M, backward=case["op"] == "backward")
    return st


def _prepare_step(case, g):
    """Each group's matrices in one buffer, each from a multiple of 8
    elements (the elements between them are zero and stay so).  Gradients and
    momenta: a few strong directions and noise, as over batches of tokens."""
    count, s = case["count"], case["s"]
    st = {"case": case, "groups": []}
    for rows, cols in ((s, case["la"]), (case["lb"], s)):
        room = _up8(rows * cols)
        few = min(4, s)
        left, right = _normal(g, count, rows, few), _normal(g, count, few, cols)

        def like(noise):
            x = torch.bmm(left, right) * 0.3 + noise * _normal(g, count, rows, cols)
            flat = torch.zeros(count, room, device="cuda")
            flat[:, :rows * cols] = x.reshape(count, rows * cols) * 1e-3
            return flat

        grad, m = like(0.5), like(0.2) * 4.0
        p = torch.zeros(count, room, device="cuda")
        p[:, :rows * cols] = _normal(g, count, rows * cols) * 0.02
        st["groups"].append({"rows": rows, "cols": cols, "room": room, "m": m,
                             "g": grad.to(torch.bfloat16) if case["g_half"] else grad,
                             "p": p.to(torch.bfloat16) if case["p_half"] else p,
                             "master": p if case["master"] else None})
    if own:
        import sparse_rank_linear_amd as srl

        def views(key):
            if st["groups"][0][key] is None:
                return None
            return [q[key][i, :q["rows"] * q["cols"]].view(q["rows"], q["cols"]) for q in st["groups"]
                    for i in range(count)]

        st["plan"] = srl.muon_plan(views("p"), views("g"), views("m"), master=views("master"))
    return st


# ---- the package's operators ----

def _own(st):
    import sparse_rank_linear_amd as srl
    case = st["case"]
    if case["op"] == "step":
        srl.muon_step(st["plan"], LR, momentum=MOMENTUM, weight_decay=DECAY, eps=EPS, steps=STEPS,
                      coefficients=COEFFICIENTS)
        return [[q["p"], q["master"], q["m"]] for q in st["groups"]]
    if case["plan"]:
        srl.adapters_plan(st["ids"], case["count"], plan=st["plan"])
    if case["op"] == "forward":
        return srl.adapters_forward(st["adapters"], st["plan"], st["X"], base=st["base"], Y=st["Y"], ws=st["ws"])
    return srl.adapters_backward(st["adapters"], st["plan"], st["X"], st["dY"], base=st["base"], dX=st["dX"],
                                 dA=st["dA"], dB=st["dB"], ws=st["ws"])


# ---- the plain forms ----

def _scaled_mask(st):
    """([M][count * r], whether a token has that rank of that adapter; the
    scale of each): every adapter runs as one product, the others masked out."""
    case = st["case"]
    mine = st["ids"].long()[:, None] == torch.arange(case["count"], device="cuda")
    live = torch.arange(case["r"], device="cuda") < st["ranks"][:, None]
    return (mine[:, :, None] & live).reshape(case["M"], -1), st["scales"].repeat_interleave(case["r"])


def _adapters(st):
    case = st["case"]
    flat = case["count"] * case["r"]
    a = st["a"].float().reshape(flat, case["K"])
    b = st["b"].float().transpose(0, 1).reshape(case["N"], flat)
    keep, scale = _scaled_mask(st)
    x, base = st["X"].float(), st["base"].float()
    t = torch.where(keep, (x @ a.t()) * scale, 0.0)
    if case["op"] == "forward":
        return (base + t @ b.t()).to(torch.bfloat16)
    dy = st["dY"].float()
    grad = torch.where(keep, (dy @ b) * scale, 0.0)
    dx = (base + grad @ a).to(torch.bfloat16)
    da = (grad.t() @ x).reshape(case["count"], case["r"], case["K"])
    db = (dy.t() @ t).reshape(case["N"], case["count"], case["r"]).transpose(0, 1).contiguous()
    return dx, da, db


def _step(st):
    return [_step_group(q) for q in st["groups"]]


def _step_group(q):
    rows, cols, n = q["rows"], q["cols"], q["rows"] * q["cols"]
    grad = q["g"].float()
    q["m"].mul_(MOMENTUM).add_(grad)
    u = (grad + MOMENTUM * q["m"])[:, :n].reshape(-1, rows, cols)
    x = u if rows <= cols else u.transpose(1, 2)
    # (the norm as a sum of rows' sums: long sums of squares stay exact)
    norm = x.square().sum(2).sum(1).sqrt()
    x = (x / (norm + EPS)[:, None, None]).contiguous()
    x = _newton_schulz(x)
    o = (x if rows <= cols else x.transpose(1, 2)).reshape(-1, n)
    scale = LR * max(1.0, rows / cols) ** 0.5
    p = q["p"] if q["master"] is None else q["master"]
    new = p.float()
    new[:, :n] = new[:, :n] * (1.0 - LR * DECAY) - scale * o
    p.copy_(new)
    if q["master"] is not None:
        q["p"].copy_(new)
    return [q["p"], q["master"], q["m"]]


def _newton_schulz(x):
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return x


def run(state):
    if own:
        return _own(state)
    return _step(state) if state["case"]["op"] == "step" else _adapters(state)


def work(case):
    if case["op"] == "step":
        s, count = case["s"], case["count"]
        n = count * s * (case["la"] + case["lb"])
        each = (2 if case["g_half"] else 4) + 8 + (8 + 2 if case["master"] else 2 * (2 if case["p_half"] else 4))
        # one symmetric product of the update with itself, one with the result, the short side's products
        return {"bytes": float(n * each), "flops": float(n * (s + 1) + 2 * n * s + 2 * count * 17 * s ** 3)}
    M, K, N, n, count = (case[k] for k in ("M", "K", "N", "requests", "count"))
    ranks = _ranks(case)
    used = sorted({i % count for i in range(n) if _has_adapter(case, i)})
    # (which adapter is whose is the seed's: the mean rank stands for each)
    mean = sum(ranks) / count
    tokens = M * sum(_has_adapter(case, i) for i in range(n)) / n
    weights = 2.0 * len(used) * mean * (K + N)
    product = 2.0 * tokens * mean * (K + N)
    if case["op"] == "forward":
        return {"bytes": tokens * K * 2 + weights + M * N * 4 + M * 4, "flops": product}
    grads = 4.0 * count * case["r"] * (K + N)
    # (T and G, dA and dB, dX)
    return {"bytes": tokens * (K + N) * 2 + weights + M * K * 4 + grads + M * 4,
            "flops": 2 * product + 2.0 * tokens * mean * K}


# ---- the definitions in float64 ----

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "step":
        return _exact_step(case, st)
    ids, ranks, scales = st["ids"].tolist(), st["ranks"].tolist(), st["scales"].tolist()
    rows = {}
    for t, a in enumerate(ids):
        rows.setdefault(a, []).append(t)
    out = st["base"].double()
    back = case["op"] == "backward"
    da = torch.zeros(st["a"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(st["b"].shape, dtype=torch.float64, device="cuda")
    for a, at in rows.items():
        if a < 0:
            continue
        at = torch.tensor(at, device="cuda")
        down, up = st["a"][a, :ranks[a]].double(), st["b"][a, :, :ranks[a]].double() * scales[a]
        t = st["X"][at].double() @ down.t()
        if not back:
            out[at] += t @ up.t()
            continue
        dy = st["dY"][at].double()
        gr = dy @ up
        out[at] += gr @ down
        da[a, :ranks[a]] = gr.t() @ st["X"][at].double()
        db[a, :, :ranks[a]] = dy.t() @ (t * scales[a])
    return (out, da, db) if back else out


def _exact_step(case, st):
    """Each singular value follows its own polynomial: the update is rebuilt
    from the eigenvectors of the short side's products."""
    a, b, c = COEFFICIENTS
    got = []
    for q in st["groups"]:
        rows, cols = q["rows"], q["cols"]
        n = rows * cols
        m = MOMENTUM * q["m"].double() + q["g"].double()
        u = (q["g"].double() + MOMENTUM * m)[:, :n].reshape(-1, rows, cols)
        o = torch.empty_like(u)
        for i in range(case["count"]):
            x = u[i] if rows <= cols else u[i].t()
            x = x / (torch.linalg.vector_norm(x) + EPS)
            value, vector = torch.linalg.eigh((x @ x.t()).cpu())
            value, vector = value.cuda().clamp(min=0.0), vector.cuda()
            grow = torch.ones_like(value)               # what the singular value has been multiplied by
            for _ in range(STEPS):
                now = value * grow * grow
                grow = grow * (a + b * now + c * now * now)
            x = vector @ (grow[:, None] * (vector.t() @ x))
            o[i] = x if rows <= cols else x.t()
        p = (q["p"] if q["master"] is None else q["master"]).double()
        p[:, :n] = p[:, :n] * (1 - LR * DECAY) - LR * max(1.0, rows / cols) ** 0.5 * o.reshape(-1, n)
        got.append([p, None if q["master"] is None else p, m])
    return got
