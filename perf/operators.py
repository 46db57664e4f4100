"""Operators around the expert layers and after the adapter gradients, for
measurement: the router, the sort of tokens by expert and the way back with
their gradients, and the AdamW step.

`run` computes them in plain torch (own = False) or through the package
(own = True); `exact` holds the definitions in float64."""

import torch

own = False

# Case keys.  Routing operators: T tokens, E experts, k experts a token, D
# columns, pad trailing tokens without any expert (a padded batch).  AdamW:
# count tensors of na and nb elements in turn, the parameter's and gradient's
# types, states in 32 or 8 bits, a float master copy or none.
BLOCK = 256                      # elements per 8-bit block
TINY = 2.0 ** -100               # blocks whose largest value is below hold zeros
BETA1, BETA2, EPS, DECAY, LR, STEP = 0.9, 0.999, 1e-8, 0.01, 2e-4, 37


def listed():
    return [
        # the smallest call: one decode step of 16 tokens over 8 experts
        {"name": "route_decode", "op": "route", "T": 16, "E": 8, "k": 2, "renorm": True, "half": False, "pad": 0},
        # a training batch over 64 fine-grained experts, full-softmax weights
        {"name": "route_train", "op": "route", "T": 16384, "E": 64, "k": 6, "renorm": False, "half": False, "pad": 0},
        # its gradient, bf16 logits, ragged token count with padding
        {"name": "route_grad", "op": "route_backward", "T": 16379, "E": 64, "k": 6, "renorm": False, "half": True,
         "pad": 37},
        # 16 decode tokens to 64 experts, 2048 columns
        {"name": "dispatch_decode", "op": "dispatch", "T": 16, "E": 64, "k": 6, "D": 2048, "pad": 0},
        # a prefill of 4099 tokens (odd, some padding) to 64 experts
        {"name": "dispatch_prefill", "op": "dispatch", "T": 4099, "E": 64, "k": 6, "D": 2048, "pad": 61},
        # the gradient of a top-2 dispatch in training
        {"name": "dispatch_grad", "op": "dispatch_backward", "T": 8192, "E": 8, "k": 2, "D": 4096, "pad": 0},
        # 16 decode tokens back from 8 experts
        {"name": "combine_decode", "op": "combine", "T": 16, "E": 8, "k": 2, "D": 4096, "base": False, "pad": 0},
        # a prefill back from 64 experts, added to the shared experts' output
        {"name": "combine_prefill", "op": "combine", "T": 4099, "E": 64, "k": 6, "D": 2048, "base": True, "pad": 61},
        # the gradient of a top-2 combine in training
        {"name": "combine_grad", "op": "combine_backward", "T": 8192, "E": 8, "k": 2, "D": 4096, "pad": 0},
        # one 4096 x 4096 layer's adapter pair (rank 80)
        {"name": "adamw_layer", "op": "adamw", "count": 2, "na": 327680, "nb": 327680, "p_half": True, "g_half": False,
         "bits": 32, "master": False},
        # every adapter of 32 blocks of seven layers, with a float master copy
        {"name": "adamw_model", "op": "adamw", "count": 448, "na": 409600, "nb": 487680, "p_half": True,
         "g_half": False, "bits": 32, "master": True},
        # the adapters of one layer's 64 experts (three matrices each), 8-bit states
        {"name": "adamw8_experts", "op": "adamw", "count": 384, "na": 163840, "nb": 112640, "p_half": True,
         "g_half": False, "bits": 8, "master": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "dispatch", "dispatch_backward", "combine", "combine_backward",
                     "adamw", "adamw"])
    if op == "adamw":
        count = _log(rng, 1, 400)
        na, nb = (_log(rng, 64, max(64, min(2_000_000, 60_000_000 // count))) for _ in range(2))
        p_half, bits = rng.random() < 0.7, rng.choice([8, 32])
        return {"op": op, "count": count, "na": na, "nb": nb, "p_half": p_half, "g_half": rng.random() < 0.4,
                "bits": bits, "master": p_half and rng.random() < 0.5}
    E = rng.choice([2, 5, 8, 16, 40, 60, 64, 128, 160, 256])
    k = rng.randint(1, min(E, 8))
    T = _log(rng, 1, 16384)
    pad = rng.choice([0, 0, T // 9])
    case = {"op": op, "T": T, "E": E, "k": k, "pad": pad}
    if op.startswith("route"):
        case.update(renorm=rng.random() < 0.5, half=rng.random() < 0.5)
        return case
    # (columns in eights, as the expert layers take them; at most 2^27 routed values)
    case["D"] = 8 * _log(rng, 8, max(8, min(1024, (1 << 24) // (T * k))))
    if op == "combine":
        case["base"] = rng.random() < 0.5
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _logits(case, g):
    """Router logits with some experts preferred, as a trained router has."""
    x = _normal(g, case["T"], case["E"]) + 0.7 * _normal(g, case["E"])
    if case["pad"]:
        x[case["T"] - case["pad"]:] = float("-inf")   # a padded token goes nowhere
    return x


def _choose(logits, k):
    """ids of the k largest logits, ties to the lowest expert, -1 for -inf."""
    vals, order = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    return torch.where(vals[:, :k] > float("-inf"), order[:, :k], -1).to(torch.int32)


def _sorted_slots(ids, E):
    """(offsets, rows, order): the stable order of the slots by expert."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    bound = torch.arange(E + 1, device=ids.device)
    offsets = torch.searchsorted(key[order], bound)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    rows = torch.where(key < E, place, -1).reshape(ids.shape)
    return offsets.to(torch.int32), rows.to(torch.int32), order


def _round8(x):
    """x [blocks][256] as e4m3 codes and scales, one scale a block."""
    top = x.abs().amax(1, keepdim=True)
    live = top >= TINY
    safe = torch.where(live, top, torch.ones_like(top))
    q = torch.where(live, x * (448.0 / safe), torch.zeros_like(x))
    return q, torch.where(live, top / 448.0, torch.zeros_like(top))


def _store_m(m):
    q, scale = _round8(m.reshape(-1, BLOCK))
    return q.to(torch.float8_e4m3fn).reshape(-1), scale.reshape(-1)


def _store_s(s):
    q, scale = _round8(s.reshape(-1, BLOCK))
    q = torch.where(q > 0, q.clamp(min=2.0 ** -9), q)   # a value above zero never codes zero
    return q.to(torch.float8_e4m3fn).reshape(-1), scale.reshape(-1)


def _sizes(case):
    return [case["na"] if i % 2 == 0 else case["nb"] for i in range(case["count"])]


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, g)
    T, E, k = case["T"], case["E"], case["k"]
    logits = _logits(case, g)
    st = {"case": case}
    if case["op"].startswith("route"):
        st["logits"] = logits.to(torch.bfloat16) if case["half"] else logits
        st["ids"] = _choose(st["logits"], k)
        st["weights"] = torch.empty(T, k, device="cuda")
        st["dweights"] = _normal(g, T, k)
        st["dlogits"] = torch.empty_like(st["logits"])
        return st
    D, n = case["D"], T * k
    ids = _choose(logits, k)
    offsets, rows, order = _sorted_slots(ids, E)
    st["ids"] = ids
    half = lambda *s: _normal(g, *s).to(torch.bfloat16)  # noqa: E731
    if case["op"] == "dispatch":
        st.update(X=half(T, D), Xs=torch.zeros(n, D, dtype=torch.bfloat16, device="cuda"),
                  offsets=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                  rows=torch.empty(T, k, dtype=torch.int32, device="cuda"),
                  slots=torch.full((n,), -1, dtype=torch.int32, device="cuda"))
        if own:
            import sparse_rank_linear_amd as srl
            st["ws"] = srl.moe_dispatch_workspace(T, k, E)
        return st
    st["rows"] = rows
    w = torch.softmax(logits.nan_to_num(neginf=0.0), -1)
    st["weights"] = torch.gather(w, 1, ids.clamp(min=0).long())
    if case["op"] in ("combine", "dispatch_backward"):
        st["Ys"] = half(n, D)
        st["Y"] = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
        st["base"] = half(T, D) if case.get("base") else None
    else:
        st.update(dY=half(T, D), Ys=half(n, D), offsets=offsets, slots=order.to(torch.int32),
                  dYs=torch.zeros(n, D, dtype=torch.bfloat16, device="cuda"),
                  dweights=torch.empty(T, k, device="cuda"))
    return st


def _prepare_adamw(case, g):
    """Tensors as views of flat buffers, each from a multiple of 256
    elements (the elements between them are zero and stay so)."""
    n = _sizes(case)
    room = [-(-s // BLOCK) * BLOCK for s in n]
    start = [sum(room[:i]) for i in range(len(n))]
    N = sum(room)
    live = torch.zeros(N, dtype=torch.bool, device="cuda")
    size = torch.empty(N, device="cuda")     # each tensor's own gradient size
    level = 10.0 ** (-5 + 3 * torch.rand(len(n), generator=torch.Generator().manual_seed(int(case["count"]))))
    for i, s in enumerate(n):
        live[start[i]:start[i] + s] = True
        size[start[i]:start[i] + room[i]] = float(level[i])
    size = torch.where(live, size, torch.zeros_like(size))
    grad = _normal(g, N) * size
    m = _normal(g, N) * size * 0.3
    v = (_normal(g, N) * size).square() * 0.5 + (0.2 * size).square()
    p = torch.where(live, _normal(g, N) * 0.01, torch.zeros_like(size))
    st = {"case": case, "g": grad.to(torch.bfloat16) if case["g_half"] else grad,
          "p": p.to(torch.bfloat16) if case["p_half"] else p, "master": p if case["master"] else None,
          "m_scale": None, "v_scale": None}
    if case["bits"] == 8:
        st["m"], st["m_scale"] = _store_m(m)
        st["v"], st["v_scale"] = _store_s(v.sqrt())
    else:
        st["m"], st["v"] = m, v
    if own:
        import sparse_rank_linear_amd as srl
        views = lambda t, d=1: None if t is None else [  # noqa: E731
            t[a // d:a // d + -(-s // d)] for a, s in zip(start, n)]
        st["plan"] = srl.adamw_plan(views(st["p"]), views(st["g"]), views(st["m"]), views(st["v"]),
                                    m_scale=views(st["m_scale"], BLOCK), v_scale=views(st["v_scale"], BLOCK),
                                    master=views(st["master"]))
    return st


# ---- the package's operators ----

def _own(st):
    import sparse_rank_linear_amd as srl
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        srl.moe_route(st["logits"], case["k"], renorm=case["renorm"], ids=st["ids"], weights=st["weights"])
        return st["ids"], st["weights"]
    if op == "route_backward":
        return srl.moe_route_backward(st["logits"], st["ids"], st["dweights"], renorm=case["renorm"],
                                      dlogits=st["dlogits"])
    if op == "dispatch":
        srl.moe_dispatch(st["ids"], case["E"], st["X"], Xs=st["Xs"], offsets=st["offsets"], rows=st["rows"],
                         slots=st["slots"], ws=st["ws"])
        return st["Xs"], st["offsets"], st["rows"], st["slots"]
    if op == "dispatch_backward":
        return srl.moe_dispatch_backward(st["Ys"], st["rows"], dX=st["Y"])
    if op == "combine":
        return srl.moe_combine(st["Ys"], st["rows"], st["weights"], base=st["base"], Y=st["Y"])
    if op == "combine_backward":
        srl.moe_combine_backward(st["dY"], st["Ys"], st["rows"], st["weights"], dYs=st["dYs"],
                                 dweights=st["dweights"])
        return st["dYs"], st["dweights"]
    srl.adamw_step(st["plan"], STEP, LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY)
    return [st[key] for key in ("p", "master", "m", "v", "m_scale", "v_scale")]


# ---- the plain forms ----

def _route(st):
    case, k = st["case"], st["case"]["k"]
    x = st["logits"].float()
    vals, order = torch.sort(x, dim=-1, descending=True, stable=True)
    chosen = vals[:, :k] > float("-inf")
    top = torch.where(vals[:, :1] > float("-inf"), vals[:, :1], torch.zeros_like(vals[:, :1]))
    e = torch.where(chosen, torch.exp(vals[:, :k] - top), 0.0)
    total = e.sum(-1, keepdim=True) if case["renorm"] else torch.exp(x - top).sum(-1, keepdim=True)
    w = torch.where(chosen, e / total, 0.0)
    return torch.where(chosen, order[:, :k], -1).to(torch.int32), w


def _route_backward(st):
    case = st["case"]
    x, ids, dw = st["logits"].float(), st["ids"].long(), st["dweights"]
    chosen, at = ids >= 0, ids.clamp(min=0)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
    ek = torch.where(chosen, torch.gather(e, 1, at), 0.0)
    total = (ek if case["renorm"] else e).sum(-1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    w, dw = ek / total, torch.where(chosen, dw, 0.0)
    mean = (w * dw).sum(-1, keepdim=True)
    out = torch.zeros_like(x) if case["renorm"] else -(e / total) * mean
    out.scatter_add_(1, at, w * (dw - mean) if case["renorm"] else w * dw)
    return out.to(st["logits"].dtype)


def _dispatch(st):
    case = st["case"]
    offsets, rows, order = _sorted_slots(st["ids"], case["E"])
    routed = torch.arange(order.numel(), device="cuda") < offsets[-1]
    slots = torch.where(routed, order.to(torch.int32), st["slots"])
    return torch.where(routed[:, None], st["X"][order // case["k"]], st["Xs"]), offsets, rows, slots


def _gathered(st):
    """Each slot's row in float [T][k][D], zero where it has none."""
    rows = st["rows"].long()
    y = st["Ys"][rows.clamp(min=0)].float()
    return torch.where((rows >= 0)[..., None], y, 0.0)


def _combine(st, weighted):
    y = _gathered(st)
    if weighted:
        y = y * torch.where(st["rows"] >= 0, st["weights"], 0.0)[..., None]
    y = y.sum(1)
    if st["base"] is not None:
        y = st["base"].float() + y
    return y.to(torch.bfloat16)


def _combine_backward(st):
    dw = (st["dY"].float()[:, None, :] * _gathered(st)).sum(-1)
    slots = st["slots"].long()
    routed = torch.arange(slots.numel(), device="cuda") < st["offsets"][-1]
    d = st["dY"][slots // st["case"]["k"]].float() * st["weights"].reshape(-1)[slots][:, None]
    return torch.where(routed[:, None], d.to(torch.bfloat16), st["dYs"]), dw


def _adamw(st):
    case = st["case"]
    g = st["g"].float()
    p = st["master"] if case["master"] else st["p"].float()
    if case["bits"] == 8:
        m = (st["m"].float().reshape(-1, BLOCK) * st["m_scale"][:, None]).reshape(-1)
        v = (st["v"].float().reshape(-1, BLOCK) * st["v_scale"][:, None]).reshape(-1).square()
    else:
        m, v = st["m"], st["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    s = v.sqrt()
    rate = LR / (1.0 - BETA1 ** STEP)
    p = p * (1.0 - LR * DECAY) - (m / (s * (1.0 - BETA2 ** STEP) ** -0.5 + EPS)) * rate
    if case["bits"] == 8:
        m, st["m_scale"] = _store_m(m)
        v, st["v_scale"] = _store_s(s)
    # the step updates what the program keeps
    st["p"], st["master"], st["m"], st["v"] = p.to(st["p"].dtype), p if case["master"] else None, m, v
    return [st[key] for key in ("p", "master", "m", "v", "m_scale", "v_scale")]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "route":
        return _route(state)
    if op == "route_backward":
        return _route_backward(state)
    if op == "dispatch":
        return _dispatch(state)
    if op == "dispatch_backward":
        return _combine(state, False)
    if op == "combine":
        return _combine(state, True)
    if op == "combine_backward":
        return _combine_backward(state)
    return _adamw(state)


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        p, g, state = (2 if case["p_half"] else 4), (2 if case["g_half"] else 4), (2 if case["bits"] == 8 else 8)
        each = g + 2 * state + (8 + p if case["master"] else 2 * p) + (16.0 / BLOCK if case["bits"] == 8 else 0)
        return {"bytes": n * each, "flops": 16.0 * n}
    T, E, k = case["T"], case["E"], case["k"]
    n, live = T * k, (T - case["pad"]) * k
    if op.startswith("route"):
        each = 2 if case["half"] else 4
        if op == "route":
            return {"bytes": T * E * each + n * 8, "flops": 3.0 * T * E}
        read = n if case["renorm"] else T * E
        return {"bytes": read * each + T * E * each + n * 8, "flops": 6.0 * T * E}
    row = 2 * case["D"]
    if op == "dispatch":
        return {"bytes": (T - case["pad"]) * row + live * row + n * 4 + n * 4 + live * 4 + (E + 1) * 4,
                "flops": 1.0 * n}
    if op == "combine_backward":
        return {"bytes": (T - case["pad"]) * row + 2 * live * row + n * 12, "flops": 3.0 * live * case["D"]}
    weighted = op == "combine"
    return {"bytes": live * row + T * row * (2 if case.get("base") else 1) + n * (8 if weighted else 4),
            "flops": (2.0 if weighted else 1.0) * live * case["D"]}


# ---- the definitions in float64 ----

def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "dispatch":
        ids = st["ids"].reshape(-1).long()
        near = [torch.nonzero(ids == e).reshape(-1) for e in range(case["E"])]   # each expert's slots, in order
        Xs, slot = torch.zeros(st["Xs"].shape, dtype=torch.float64, device="cuda"), torch.cat(near)
        Xs[:slot.numel()] = st["X"][slot // case["k"]].double()
        return [Xs, None, None, None]
    if op == "adamw":
        return _exact_adamw(case, st)
    if op.startswith("route"):
        x = st["logits"].double()
        prob = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)       # (a row of -inf: nothing)
        ids = st["ids"].long()
        hot = torch.nn.functional.one_hot(ids + 1, case["E"] + 1)[..., 1:].double()   # [T][k][E]
        w = (hot * prob[:, None, :]).sum(-1)
        norm = w.sum(-1, keepdim=True)
        if case["renorm"]:
            w = torch.where(norm > 0, w / norm, torch.zeros_like(w))
        if op == "route":
            return [None, w]
        dw = st["dweights"].double()
        up = (hot * dw[..., None]).sum(1)                             # dL/dw by expert
        if case["renorm"]:
            prob = (hot * w[..., None]).sum(1)                        # the softmax over the chosen
        return prob * (up - (prob * up).sum(-1, keepdim=True))
    T, k, D = case["T"], case["k"], case["D"]
    slot = torch.arange(T * k, device="cuda")
    row = st["rows"].reshape(-1).long()
    slot, row = slot[row >= 0], row[row >= 0]                         # (slot, row) of every routed pair
    w = st["weights"].double().reshape(-1)[slot]
    if op == "combine_backward":
        dYs = torch.zeros(T * k, D, dtype=torch.float64, device="cuda")
        dYs[row] = w[:, None] * st["dY"][slot // k].double()
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        for a in range(0, slot.numel(), 1 << 14):
            s, r = slot[a:a + (1 << 14)], row[a:a + (1 << 14)]
            dw[s] = (st["dY"][s // k].double() * st["Ys"][r].double()).sum(-1)
        return [dYs, dw.reshape(T, k)]
    y = torch.zeros(T, D, dtype=torch.float64, device="cuda") if st["base"] is None else st["base"].double()
    by_rank = slot % k
    for j in range(k):
        t, r = slot[by_rank == j] // k, row[by_rank == j]
        part = st["Ys"][r].double()
        y[t] += part * w[by_rank == j][:, None] if op == "combine" else part
    return y


def _exact_adamw(case, st):
    g = st["g"].double()
    small = case["bits"] == 8
    m = st["m"].double()
    v = st["v"].double()
    if small:
        m = m * st["m_scale"].double().repeat_interleave(BLOCK)
        v = (v * st["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    p = (st["master"] if case["master"] else st["p"]).double()
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS)
    if not small:
        return [p, p if case["master"] else None, m, v, None, None]
    blocks = [x.reshape(-1, BLOCK) for x in (m, v.sqrt())]
    ms, vs = (x.abs().amax(1) / 448 for x in blocks)
    m8, s8 = (_e4m3(x / torch.where(a > 0, a, torch.ones_like(a))[:, None]) for x, a in zip(blocks, (ms, vs)))
    s8 = torch.where(blocks[1] > 0, s8.clamp(min=2.0 ** -9), s8)
    return [p, p if case["master"] else None, m8.reshape(-1), s8.reshape(-1), ms, vs]


def _e4m3(x):
    """The value of the format nearest to x (ties to even): 3 bits after the
    first, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step
