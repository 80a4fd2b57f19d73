"""Group-limited routing and low-rank adapters, each with its gradient: cases, plain forms, framework calls.

Four operators of a 4-bit MoE layer that is served to many requests and fine-tuned:

``route``          logits -> the k experts of each token, picked from its best groups of experts by score + bias, and
                   their weights (softmax or sigmoid scores, renormalised or not, times a scale).
``route_grad``     the gradient of those weights in the logits.
``adapters``       out = base + s_l (x A_l^T) B_l, every sequence of rows with the adapter l of its request, or none.
``adapters_grad``  the gradients of that in x, A and B.
"""
import math

import numpy as np
import torch

own = False


def listed():
    return [
        # one token of a sigmoid router with a balance bias, 8 groups of 16 experts: latency
        dict(name="route_T1", op="route", T=1, E=128, k=8, n_group=8, topk_group=4, sigmoid=True, bias=True, group_max=False,
             renorm=True, masked=0.0, dtype="fp32"),
        # a decode batch, softmax scores, the best expert stands for its group, bf16 logits (ties)
        dict(name="route_T64_bf16", op="route", T=64, E=512, k=10, n_group=16, topk_group=4, sigmoid=False, bias=False,
             group_max=True, renorm=False, masked=0.0, dtype="bf16"),
        # a training batch with padding
        dict(name="route_T16384", op="route", T=16384, E=512, k=10, n_group=8, topk_group=4, sigmoid=True, bias=True,
             group_max=False, renorm=True, masked=0.05, dtype="fp32"),
        # the gradient of a micro-batch
        dict(name="route_grad_T255", op="route_grad", T=255, E=288, k=8, sigmoid=True, renorm=True, masked=0.1, dtype="fp32"),
        # the gradient of a training batch of an odd size, weights that are not renormalised: every logit gets one
        dict(name="route_grad_T30011", op="route_grad", T=30011, E=288, k=8, sigmoid=False, renorm=False, masked=0.0,
             dtype="bf16"),
        # one token of one request beside a square projection: latency
        dict(name="adapters_T1", op="adapters", T=1, K=2048, N=2048, R=16, L=8, kind="rows", n_seq=1, none=0.0, out="bf16"),
        # a decode batch, most requests with an adapter of their own: weight streaming
        dict(name="adapters_T64_decode", op="adapters", T=64, K=2048, N=4096, R=16, L=64, kind="rows", n_seq=64, none=0.1,
             out="bf16"),
        # decoding requests and a few prompts in one batch, odd sizes, fp32 results
        dict(name="adapters_T1001_mixed", op="adapters", T=1001, K=1416, N=1000, R=24, L=12, kind="mixed", n_seq=40, none=0.1,
             out="fp32"),
        # prompts: the rows' bytes
        dict(name="adapters_T4096_prompt", op="adapters", T=4096, K=2048, N=4096, R=64, L=4, kind="packed", n_seq=3, none=0.0,
             out="bf16"),
        # one short training sequence
        dict(name="adapters_grad_T300", op="adapters_grad", T=300, K=2048, N=2048, R=8, L=1, kind="packed", n_seq=1, none=0.0,
             base=False),
        # a training batch of packed sequences for three adapters, added to the projection's own gradient
        dict(name="adapters_grad_T8192", op="adapters_grad", T=8192, K=2048, N=4096, R=32, L=3, kind="packed", n_seq=11,
             none=0.0, base=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "adapters", "adapters", "adapters_grad"])
    if op in ("route", "route_grad"):
        n_group = rng.choice([1, 2, 4, 8, 8, 16, rng.randint(1, 32)])
        E = n_group * max(2, _log(rng, 16, 1024) // n_group)
        T = _log(rng, 1, min(60000, (1 << 23) // E))
        case = dict(op=op, T=T, E=E, sigmoid=rng.random() < 0.5, renorm=rng.random() < 0.7, masked=rng.choice([0.0, 0.0, 0.1]),
                    dtype=rng.choice(["fp32", "fp32", "bf16"]))
        if op == "route_grad":
            return dict(case, k=rng.randint(1, min(16, E)))
        topk_group = rng.randint(1, n_group)
        return dict(case, k=rng.randint(1, min(16, topk_group * (E // n_group))), n_group=n_group, topk_group=topk_group,
                    bias=rng.random() < 0.6, group_max=rng.random() < 0.3)
    kind = rng.choice(["rows", "mixed", "packed"])
    R = rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 128)])
    K, N = 8 * _log(rng, 32, 512), 8 * _log(rng, 32, 512)
    most = (1 << 25) // (K + N)
    T = _log(rng, 1, max(2, min(256, most))) if kind == "rows" else _log(rng, 2, max(3, most))
    n_seq = T if kind == "rows" else _log(rng, 1, max(2, min(100, T // 2)))
    L = _log(rng, 1, max(2, min(64, (1 << 25) // (R * (K + N)))))
    case = dict(op=op, T=T, K=K, N=N, R=R, L=L, kind=kind, n_seq=n_seq, none=rng.choice([0.0, 0.0, 0.2]))
    if op == "adapters":
        return dict(case, out=rng.choice(["bf16", "bf16", "fp32"]))
    return dict(case, base=rng.random() < 0.5)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 29)
    return g


def _lengths(kind, T, n, r):
    """Lengths of n sequences of T rows: one row each, ragged ones, or decoding requests before a few prompts."""
    if kind == "rows":
        return np.ones(T, np.int64)
    lead = 0 if kind == "packed" else min(n - max(1, n // 10), T - 1)
    cuts = np.sort(r.integers(0, T - lead + 1, n - lead - 1))
    if len(cuts) >= 3:
        cuts[1] = cuts[0]  # an empty sequence
    return np.concatenate([np.ones(lead, np.int64), np.diff(np.concatenate([[0], cuts, [T - lead]]))])


def _acts(T, H, g):
    """Activations ~N(0, 1) with a few channels an order of magnitude larger, as a residual stream has."""
    gain = torch.ones(H, device="cuda")
    gain[torch.randint(0, H, (max(1, H // 256),), device="cuda", generator=g)] = 12.0
    return (torch.randn(T, H, device="cuda", generator=g) * gain).to(torch.bfloat16)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    T = case["T"]
    if op in ("route", "route_grad"):
        E, k = case["E"], case["k"]
        popular = torch.randn(E, device="cuda", generator=g) * 0.5
        logits = (torch.randn(T, E, device="cuda", generator=g) * 1.5 + popular).to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
        mask = torch.rand(T, device="cuda", generator=g) >= case["masked"] if case["masked"] > 0 else None
        if mask is not None:
            logits = torch.where(mask[:, None], logits, float("nan"))  # what a padded row holds is anybody's guess
        st = dict(op=op, logits=logits, k=k, sigmoid=case["sigmoid"], renorm=case["renorm"], scale=2.5)
        if op == "route_grad":
            ids = torch.rand(T, E, device="cuda", generator=g).add_(logits.float().nan_to_num()).topk(k, dim=1).indices.to(torch.int32)
            st["ids"] = ids if mask is None else torch.where(mask[:, None], ids, -1)
            st["grad_w"] = torch.randn(T, k, device="cuda", generator=g) * 0.01
            return st
        # a balance bias is the sum of many steps of one size
        bias = torch.round(-popular * 100).mul_(0.001) if case["bias"] else None
        return dict(st, mask=mask, bias=bias, n_group=case["n_group"], topk_group=case["topk_group"], group_max=case["group_max"])
    K, N, R, L = (case[v] for v in ("K", "N", "R", "L"))
    r = np.random.default_rng(int(seed) + 7)
    lengths = _lengths(case["kind"], T, case["n_seq"], r)
    starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    ids = r.integers(0, L, len(lengths)).astype(np.int32)
    ids[r.random(len(lengths)) < case["none"]] = -1
    a = (torch.randn(L, R, K, device="cuda", generator=g) * K ** -0.5).to(torch.bfloat16)
    b = (torch.randn(L, R, N, device="cuda", generator=g) * 0.02).to(torch.bfloat16)
    scale = torch.rand(L, device="cuda", generator=g) * 2 + 0.5
    x = _acts(T, K, g)
    st = dict(op=op, x=x, a=a, b=b, scale=scale, ids=torch.from_numpy(ids).cuda(), lengths=lengths, host_ids=ids,
              starts=None if case["kind"] == "rows" else torch.from_numpy(starts).cuda())
    if op == "adapters":
        st["base"] = torch.randn(T, N, device="cuda", generator=g).to(torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    else:
        st["dy"] = (torch.randn(T, N, device="cuda", generator=g) * 0.01).to(torch.bfloat16)
        st["base"] = (torch.randn(T, K, device="cuda", generator=g) * 0.01).to(torch.bfloat16) if case["base"] else None
        st["kept"] = _shrink(x, a, scale, _spans(lengths, ids))  # the forward pass keeps it
    if own:
        import expert_slot_cache_gb300 as M
        st["adapters"] = M.Adapters(a, b, scale)
    return st


def _spans(lengths, ids):
    end = np.cumsum(lengths)
    return [(int(e - n), int(e), int(i)) for n, e, i in zip(lengths, end, ids) if n > 0 and i >= 0]


def _shrink(x, w, scale, spans):
    """s_l x W_l^T of every row, fp32."""
    v = torch.zeros(x.shape[0], w.shape[1], device=x.device)
    for t0, t1, l in spans:
        v[t0:t1] = scale[l] * (x[t0:t1].float() @ w[l].float().T)
    return v


def _expand(v, w, base, spans, like, dtype):
    out = torch.zeros(v.shape[0], w.shape[2], device=v.device) if base is None else base.float()
    for t0, t1, l in spans:
        out[t0:t1] += v[t0:t1] @ w[l].float()
    return out.to(dtype)


def _plain_rows(st):
    """One row to a sequence: gathered weights, one batched product each way."""
    l = st["ids"].long().clamp(min=0)
    v = torch.bmm(st["a"][l].float(), st["x"].float()[:, :, None])
    v = v * torch.where(st["ids"] >= 0, st["scale"][l], 0.0)[:, None, None]
    return (st["base"].float() + torch.bmm(v.transpose(1, 2), st["b"][l].float())[:, 0]).to(st["base"].dtype)


def _plain_adapters(st):
    if st["starts"] is None and st["op"] == "adapters":
        return _plain_rows(st)
    spans = _spans(st["lengths"], st["host_ids"])
    if st["op"] == "adapters":
        return _expand(_shrink(st["x"], st["a"], st["scale"], spans), st["b"], st["base"], spans, st["x"], st["base"].dtype)
    dy, x = st["dy"], st["x"]
    dv = _shrink(dy, st["b"], st["scale"], spans)
    da = torch.zeros(st["a"].shape, device=x.device)
    db = torch.zeros(st["b"].shape, device=x.device)
    for t0, t1, l in spans:
        da[l] += dv[t0:t1].T @ x[t0:t1].float()
        db[l] += st["kept"][t0:t1].T @ dy[t0:t1].float()
    return dict(dx=_expand(dv, st["a"], st["base"], spans, x, torch.bfloat16), da=da, db=db)


def _plain_route(st):
    logits, k, G = st["logits"], st["k"], st["n_group"]
    T, E = logits.shape
    # choices next to each other need 64 bits
    l = logits.double()
    if st["mask"] is not None:
        l = torch.where(st["mask"][:, None], l, 0.0)
    e = torch.exp(l - l.max(1, keepdim=True).values)
    s = 1 / (1 + torch.exp(-l)) if st["sigmoid"] else e / e.sum(1, keepdim=True)
    c = l if st["bias"] is None else s + st["bias"].double()
    if G > 1:
        grouped = (s if st["bias"] is None and not st["group_max"] else c).view(T, G, E // G)
        best = grouped.max(2).values if st["group_max"] or E == G else torch.topk(grouped, 2, dim=2).values.sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :st["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        c = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), c, float("-inf"))
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids).float()
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * st["scale"]
    ids = ids.to(torch.int32)
    if st["mask"] is not None:
        ids, w = torch.where(st["mask"][:, None], ids, -1), torch.where(st["mask"][:, None], w, 0.0)
    return dict(ids=ids, w=w)


def _route_grad(st, dtype):
    T, E = st["logits"].shape
    valid = st["ids"] >= 0
    ids, g = st["ids"].clamp(min=0).long(), torch.where(valid, st["grad_w"], 0.0).to(dtype) * st["scale"]
    l = torch.where(valid[:, :1], st["logits"].to(dtype), 0.0)
    grad = torch.zeros(T, E, dtype=dtype, device=l.device)
    if st["sigmoid"]:
        p = 1 / (1 + torch.exp(-l.gather(1, ids)))
        jac = 1 - p
    else:
        lk = l.gather(1, ids) if st["renorm"] else l
        p = torch.exp(lk - lk.max(1, keepdim=True).values)
        jac = 1.0
    if st["renorm"]:
        p = p / p.sum(1, keepdim=True)
        return grad.scatter_add_(1, ids, p * (g - (p * g).sum(1, keepdim=True)) * jac)
    if st["sigmoid"]:
        return grad.scatter_add_(1, ids, p * g * jac)
    p = p / p.sum(1, keepdim=True)
    grad.scatter_add_(1, ids, g)
    return p * (grad - (p * grad).sum(1, keepdim=True))


def run(state):
    op = state["op"]
    if own:
        import expert_slot_cache_gb300 as M
        if op == "route":
            return M.route_groups(state["logits"], state["k"], state["n_group"], state["topk_group"], sel_bias=state["bias"],
                                  token_mask=state["mask"], sigmoid=state["sigmoid"], group_max=state["group_max"],
                                  renormalise=state["renorm"], scale=state["scale"])._asdict()
        if op == "route_grad":
            return M.route_groups_grad(state["logits"], state["ids"], state["grad_w"], sigmoid=state["sigmoid"],
                                       renormalise=state["renorm"], scale=state["scale"])
        if op == "adapters":
            # fp32 results of sequences are added in place, as the plain form adds them
            place = state["base"] if state["starts"] is not None and state["base"].dtype == torch.float32 else None
            return state["adapters"].forward(state["x"], state["ids"], base=state["base"], seq_start=state["starts"], out=place)
        return state["adapters"].grad(state["dy"], state["x"], state["kept"], state["ids"], base=state["base"],
                                      seq_start=state["starts"])._asdict()
    if op == "route":
        return _plain_route(state)
    if op == "route_grad":
        return _route_grad(state, torch.float32).to(state["logits"].dtype)
    return _plain_adapters(state)


def work(case):
    op, T = case["op"], case["T"]
    if op in ("route", "route_grad"):
        E, k, b = case["E"], case["k"], 4 if case["dtype"] == "fp32" else 2
        if op == "route":
            return dict(bytes=T * E * b + 8 * T * k + (4 * E if case["bias"] else 0), flops=6 * T * E)
        dense = not case["sigmoid"] and not case["renorm"]
        return dict(bytes=T * E * b * (2 if dense else 1) + (8 + (0 if dense else b)) * T * k, flops=(6 if dense else 1) * T * E + 10 * T * k)
    K, N, R, L, n = (case[v] for v in ("K", "N", "R", "L", "n_seq"))
    used = L * (1 - (1 - 1 / L) ** (n * (1 - case["none"])))  # expected number of adapters in use
    weights = used * R * (K + N)
    rows = T * (1 - case["none"])
    if op == "adapters":
        return dict(bytes=2 * rows * K + 2 * weights + T * N * (8 if case["out"] == "fp32" else 4), flops=2 * rows * R * (K + N))
    return dict(bytes=2 * T * (K + N) + (4 if case["base"] else 2) * T * K + 4 * T * R + 2 * weights + 4 * L * R * (K + N),
                flops=4 * rows * R * (K + N))


def exact(case, seed):
    """The definitions in 64 bits, token by token in numpy or sequence by sequence."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    F = torch.float64
    if st["op"] == "route":
        if case["T"] > 20000:
            return None
        return _exact_route(st)
    if st["op"] == "route_grad":
        # the Jacobian of the weights, written out by the quotient rule
        l, scale = st["logits"].to(F), st["scale"]
        T, E = l.shape
        rows = torch.nonzero(st["ids"][:, 0] >= 0)[:, 0]
        ids, g = st["ids"][rows].long(), st["grad_w"][rows].to(F)
        one = torch.zeros(len(rows), E, dtype=F, device="cuda").scatter_(1, ids, g * scale)  # d / d s_e, not renormalised
        on = torch.zeros_like(one).scatter_(1, ids, 1.0)
        if st["sigmoid"]:
            s = torch.sigmoid(l[rows])
        else:
            s = torch.softmax(l[rows], 1)
        if st["renorm"]:
            total = (s * on).sum(1, keepdim=True)
            one = (one - on * (one * s).sum(1, keepdim=True) / total) / total
        grad = torch.zeros(T, E, dtype=F, device="cuda")
        grad[rows] = s * (1 - s) * one if st["sigmoid"] else s * (one - (s * one).sum(1, keepdim=True))
        return grad
    x, a, b, scale = st["x"].to(F), st["a"].to(F), st["b"].to(F), st["scale"].to(F)
    first = 0
    if st["op"] == "adapters":
        out = st["base"].to(F)
        for n, l in zip(st["lengths"].tolist(), st["host_ids"].tolist()):
            if n and l >= 0:
                out[first:first + n] += torch.linalg.multi_dot([x[first:first + n], a[l].T, b[l]]) * scale[l] if n > 1 else \
                    (x[first:first + 1] @ a[l].T) @ b[l] * scale[l]
            first += n
        return out
    dy = st["dy"].to(F)
    dx = torch.zeros_like(x) if st["base"] is None else st["base"].to(F)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for n, l in zip(st["lengths"].tolist(), st["host_ids"].tolist()):
        if n and l >= 0:
            xs, ys = x[first:first + n], dy[first:first + n]
            dv = (ys @ b[l].T) * scale[l]
            dx[first:first + n] += dv @ a[l]
            da[l] += dv.T @ xs
            db[l] += (xs @ a[l].T).T @ ys * scale[l]
        first += n
    return dict(dx=dx, da=da, db=db)


def _exact_route(st):
    l, k, G = st["logits"].double().cpu().numpy(), st["k"], st["n_group"]
    T, E = l.shape
    valid = np.ones(T, bool) if st["mask"] is None else st["mask"].cpu().numpy()
    bias = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in np.nonzero(valid)[0]:
        if st["sigmoid"]:
            s = 1 / (1 + np.exp(-l[t]))
        else:
            e = np.exp(l[t] - l[t].max())
            s = e / e.sum()
        c = l[t] if bias is None else s + bias
        pool = np.arange(E)
        if G > 1:
            by = (s if bias is None else c) if not st["group_max"] else c
            top = np.sort(by.reshape(G, -1), axis=1)[:, ::-1]
            score = top[:, 0] if st["group_max"] or E == G else top[:, 0] + top[:, 1]
            chosen = np.sort(np.lexsort((np.arange(G), -score))[:st["topk_group"]])
            pool = (chosen[:, None] * (E // G) + np.arange(E // G)).reshape(-1)
        ids[t] = pool[np.lexsort((pool, -c[pool]))[:k]]
        w[t] = s[ids[t]]
        if st["renorm"]:
            w[t] /= w[t].sum()
    return dict(ids=ids, w=w * st["scale"])
