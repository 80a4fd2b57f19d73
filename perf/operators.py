"""The 4-bit operators and the router's balance loss: cases, plain forms, framework calls.

Three operators of a slot-cached MoE layer:

``linear``   y = x W with 4-bit weights and one scale per group of inputs and output column
             (the projections beside the layer, the shared expert, the vocabulary head).
``experts``  out[t] = sum_j w[t][j] * ffn_{ids[t][j]}(x[t]), SwiGLU experts in 4-bit slabs.
``balance``  the router's balance loss over packed sequences, per-expert counts, and the
             gradient of the loss in the logits.

A 4-bit weight is ``(code - 8) * scale``: codes 0..15, one bf16 scale for each ``group``
consecutive inputs of one output column (the last group of a column may be short).
"""
import math

import numpy as np
import torch

own = False

# (hidden, intermediate, experts, top-k) of the framework's own layer configurations
QWEN = dict(H=2048, I=768, E=128, k=8)
FLASH = dict(H=2048, I=512, E=512, k=10)
STACK = dict(H=2048, I=512, E=288, k=8)
TINY = dict(H=256, I=128, E=16, k=2)


def listed():
    return [
        # one token through a square projection of the layer's hidden size: latency
        dict(name="linear_T1_square", op="linear", T=1, K=2048, N=2048, group=128, out="bf16"),
        # one token through a vocabulary head, an odd number of columns: pure weight streaming
        dict(name="linear_T1_head", op="linear", T=1, K=2048, N=100003, group=64, out="bf16"),
        # a few tokens, nothing a multiple of a tile or a group; fp32 results as a sampler wants them
        dict(name="linear_T5_ragged", op="linear", T=5, K=1416, N=1001, group=32, out="fp32"),
        # a decode batch of an odd size
        dict(name="linear_T33_batch", op="linear", T=33, K=4096, N=4096, group=128, out="bf16"),
        # a prompt: compute bound
        dict(name="linear_T4096_prompt", op="linear", T=4096, K=2048, N=4096, group=128, out="bf16"),
        # one token's top-8 experts of 128
        dict(name="experts_T1", op="experts", T=1, group=128, skew=0.5, **QWEN),
        # a small decode batch
        dict(name="experts_T8", op="experts", T=8, group=128, skew=0.5, **QWEN),
        # a decode batch over 288 small experts, finer groups
        dict(name="experts_T32_stack", op="experts", T=32, group=64, skew=0.0, **STACK),
        # a prompt with uneven expert loads
        dict(name="experts_T4096_prompt", op="experts", T=4096, group=128, skew=1.0, **QWEN),
        # a micro-batch of one sequence: latency
        dict(name="balance_T64", op="balance", T=64, E=128, k=8, n_seq=1, masked=0.0, sigmoid=False, dtype="fp32",
             grad=True),
        # a training batch of ragged packed sequences with padding, bf16 logits, 512 experts
        dict(name="balance_T16384_packed", op="balance", T=16384, E=512, k=10, n_seq=37, masked=0.1, sigmoid=False,
             dtype="bf16", grad=True),
        # an evaluation pass of the sigmoid router: the loss and the counts only
        dict(name="balance_T30011_sigmoid", op="balance", T=30011, E=288, k=8, n_seq=5, masked=0.0, sigmoid=True,
             dtype="fp32", grad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "experts", "balance"])
    if op == "linear":
        T = _log(rng, 1, 4096)
        K = 8 * _log(rng, 32, 1024)
        most = min(1 << 28, (1 << 35) // T) // K
        N = _log(rng, 64, max(65, min(131072, most)))
        return dict(op=op, T=T, K=K, N=N, group=rng.choice([32, 64, 128]), out=rng.choice(["bf16", "bf16", "fp32"]) if T <= 64 else "bf16")
    if op == "experts":
        shape = rng.choice([QWEN, FLASH, STACK, TINY, dict(H=64 * rng.randint(5, 32), I=32 * rng.randint(3, 24), E=rng.randint(9, 200), k=rng.randint(1, 7))])
        return dict(op=op, T=_log(rng, 1, 3000), group=rng.choice([32, 64, 128]), skew=round(rng.uniform(0.0, 1.2), 2), **shape)
    E = _log(rng, 8, 1024)
    T = _log(rng, 1, min(60000, (1 << 23) // E))
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(16, E)), n_seq=_log(rng, 1, max(2, min(200, T // 4))), masked=rng.choice([0.0, 0.0, 0.05, 0.4]),
                sigmoid=rng.random() < 0.4, dtype=rng.choice(["fp32", "fp32", "bf16"]), grad=rng.random() < 0.75)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _acts(T, H, g):
    """Activations ~N(0, 1) with a few channels an order of magnitude larger, as a residual stream has."""
    gain = torch.ones(H, device="cuda")
    gain[torch.randint(0, H, (max(1, H // 256),), device="cuda", generator=g)] = 12.0
    return (torch.randn(T, H, device="cuda", generator=g) * gain).to(torch.bfloat16)


def _codes(n, g):
    """4-bit codes of weights that are about normal, in bytes."""
    c = torch.empty(n, dtype=torch.uint8, device="cuda")
    for i in range(0, n, 1 << 27):
        m = min(1 << 27, n - i)
        c[i:i + m] = torch.randn(m, device="cuda", generator=g, dtype=torch.float16).mul_(2.4).add_(8.0).round_().clamp_(0, 15)
    return c


def _scales(shape, g):
    return (torch.randn(shape, device="cuda", generator=g).mul_(0.25).exp_() * (0.02 / 2.4)).to(torch.bfloat16)


def _groups(K, group):
    return -(-K // group)


def _profile(E, skew, xp=np):
    """A fixed popularity profile of the experts: normal quantiles times ``skew``, in a mixed order."""
    q = (np.arange(E) * 0.6180339887 + 0.31) % 1.0
    return skew * np.sqrt(2.0) * np.array([_erfinv(2 * min(max(v, 1e-3), 1 - 1e-3) - 1) for v in q])


def _erfinv(v):
    a, w = 0.147, math.log(max(1e-12, 1 - v * v))
    t = 2 / (math.pi * a) + w / 2
    return math.copysign(math.sqrt(math.sqrt(t * t - w / a) - t), v)


def _lengths(T, n, r):
    """n + 1 starts of packed sequences over T tokens: uneven, some of them empty."""
    cuts = np.sort(r.integers(0, T + 1, max(0, n - 1)))
    if n >= 4:
        cuts[1] = cuts[0]  # an empty sequence
    return np.concatenate([[0], cuts, [T]]).astype(np.int32)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "linear":
        T, K, N, group = case["T"], case["K"], case["N"], case["group"]
        x = _acts(T, K, g)
        codes = _codes(K * N, g).view(K, N)
        scales = _scales((_groups(K, group), N), g)
        st = dict(op=op, x=x, codes=codes, scales=scales, group=group, out=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
        if own:
            import expert_slot_cache_gb300 as M
            st["layer"] = M.W4Linear(M.w4_pack(codes, scales, group), K, N, group, max_tokens=T, out_dtype=st["out"])
            del st["codes"], st["scales"]
        return st
    if op == "experts":
        T, H, I, E, k, group = (case[v] for v in ("T", "H", "I", "E", "k", "group"))
        x = _acts(T, H, g)
        codes = _codes(E * 3 * H * I, g).view(E, 3 * H * I)
        scales = _scales((E, 2 * _groups(H, group) * I + _groups(I, group) * H), g)
        logits = torch.randn(T, E, device="cuda", generator=g) + torch.from_numpy(_profile(E, case["skew"])).float().cuda()
        top, ids = torch.topk(logits, k, dim=1)
        ids = ids.to(torch.int32)
        w = torch.exp(top - top[:, :1])
        w = w / w.sum(1, keepdim=True)
        e2s = torch.randperm(E, device="cuda", generator=g).to(torch.int32)  # expert -> slot of the pool
        st = dict(op=op, x=x, ids=ids, w=w, H=H, I=I, group=group, e2s=e2s)
        order = torch.empty(E, dtype=torch.int64, device="cuda")
        order[e2s.long()] = torch.arange(E, device="cuda")
        if own:
            import expert_slot_cache_gb300 as M
            pool = M.w4_pack_slabs(codes, scales, H, I, group)[order].contiguous()
            st["layer"] = M.W4Experts(pool, H, I, k, E, group, e2s=e2s, max_tokens=T)
        else:
            st["codes"], st["scales"] = codes[order], scales[order]
        return st
    T, E, k = case["T"], case["E"], case["k"]
    r = np.random.default_rng(int(seed) + 5)
    starts = _lengths(T, case["n_seq"], r)
    logits = torch.randn(T, E, device="cuda", generator=g) * 1.5 + torch.from_numpy(_profile(E, 0.7)).float().cuda()
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    mask = None
    if case["masked"] > 0:
        mask = torch.rand(T, device="cuda", generator=g) >= case["masked"]
        if case["n_seq"] >= 3:
            mask[int(starts[2]):int(starts[3])] = False  # a sequence of padding only
        logits = torch.where(mask[:, None], logits, float("nan"))  # what a padded row holds is anybody's guess
        ids = torch.where(mask[:, None], ids, -1)
    logits = logits.to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
    st = dict(op=op, logits=logits, ids=ids.contiguous(), mask=mask, starts=torch.from_numpy(starts).cuda(), coef=0.01, sigmoid=case["sigmoid"], grad=case["grad"])
    return st


def _weight(codes, scales, group, dtype):
    """(code - 8) * scale of [..., K, N] codes with [..., ceil(K / group), N] scales."""
    K = codes.shape[-2]
    s = scales.to(dtype).repeat_interleave(group, dim=-2)[..., :K, :]
    return (codes.to(dtype) - 8) * s


def _split(codes, scales, H, I, group, dtype):
    """The gate, up and down matrices of [A][...] slabs."""
    A, gh, gi = codes.shape[0], _groups(H, group), _groups(I, group)
    c, s = codes.split([H * I, H * I, I * H], 1), scales.split([gh * I, gh * I, gi * H], 1)
    shapes = [(H, I, gh), (H, I, gh), (I, H, gi)]
    return [_weight(a.reshape(A, K, N), b.reshape(A, n, N), group, dtype) for a, b, (K, N, n) in zip(c, s, shapes)]


def _plain_experts(st):
    x, ids, w, H, I, group = (st[v] for v in ("x", "ids", "w", "H", "I", "group"))
    T, k = ids.shape
    act, slot = torch.unique(ids.reshape(-1), return_inverse=True)  # the experts in use
    s = st["e2s"][act.long()].long()
    wg, wu, wd = _split(st["codes"][s], st["scales"][s], H, I, group, torch.float32)
    count = torch.bincount(slot, minlength=act.numel())
    order = torch.argsort(slot, stable=True)
    row = torch.arange(T * k, device=x.device) - (torch.cumsum(count, 0) - count)[slot[order]]
    xp = torch.zeros(act.numel(), int(count.max()), H, device=x.device)
    xp[slot[order], row] = x.float()[order // k]
    g, u = torch.bmm(xp, wg), torch.bmm(xp, wu)
    y = torch.bmm(g / (1 + torch.exp(-g)) * u, wd)
    rows = torch.empty(T * k, H, device=x.device)
    rows[order] = y[slot[order], row]
    return (rows.view(T, k, H) * w[:, :, None]).sum(1).to(torch.bfloat16)


def _balance(logits, ids, mask, starts, coef, sigmoid, grad, dtype):
    T, E = logits.shape
    k = ids.shape[1]
    n_seq = starts.numel() - 1
    valid = torch.ones(T, dtype=torch.bool, device=logits.device) if mask is None else mask
    seq = torch.searchsorted(starts[1:].contiguous(), torch.arange(T, device=starts.device, dtype=starts.dtype), right=True)
    flat = torch.where(valid[:, None], seq[:, None] * E + ids, n_seq * E).reshape(-1)
    counts = torch.bincount(flat, minlength=n_seq * E + 1)[:-1].view(n_seq, E)
    tokens = torch.bincount(torch.where(valid, seq, n_seq), minlength=n_seq + 1)[:-1]
    total = valid.sum().clamp(min=1).to(dtype)
    f = counts.to(dtype) * (E / k) / tokens.clamp(min=1).to(dtype)[:, None]
    l = torch.where(valid[:, None], logits.to(dtype), 0.0)
    e = 1 / (1 + torch.exp(-l)) if sigmoid else torch.exp(l - l.max(1, keepdim=True).values)
    p = torch.where(valid[:, None], e / e.sum(1, keepdim=True), 0.0)
    ft = f[seq]
    d = (p * ft).sum(1)
    res = dict(loss=coef * d.sum() / total, counts=counts.to(torch.int32))
    if grad:
        gr = (coef / total) * p * (ft - d[:, None])
        res["grad"] = gr * (1 - e) if sigmoid else gr
    return res


def run(state):
    op = state["op"]
    if op == "linear":
        if own:
            return state["layer"].forward(state["x"])
        return (state["x"].float() @ _weight(state["codes"], state["scales"], state["group"], torch.float32)).to(state["out"])
    if op == "experts":
        return state["layer"].forward(state["x"], state["ids"], state["w"]) if own else _plain_experts(state)
    if own:
        import expert_slot_cache_gb300 as M
        return M.balance_loss(state["logits"], state["ids"], state["coef"], seq_start=state["starts"], token_mask=state["mask"], sigmoid=state["sigmoid"],
                              with_grad=state["grad"])._asdict()
    r = _balance(state["logits"], state["ids"], state["mask"], state["starts"], state["coef"], state["sigmoid"], state["grad"], torch.float32)
    r["grad"] = r["grad"].to(state["logits"].dtype) if state["grad"] else None
    return r


def work(case):
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return dict(bytes=K * N / 2 + 2 * _groups(K, case["group"]) * N + 2 * T * K + (4 if case["out"] == "fp32" else 2) * T * N, flops=2 * T * K * N)
    if op == "experts":
        T, H, I, E, k, group = (case[v] for v in ("T", "H", "I", "E", "k", "group"))
        draws = np.random.default_rng(1).standard_normal((400, E)) + _profile(E, case["skew"])
        picked = np.zeros(E)
        np.add.at(picked, np.argpartition(-draws, k - 1, axis=1)[:, :k].reshape(-1), 1 / 400)
        active = float((1 - (1 - np.minimum(picked, 1.0)) ** T).sum())  # expected number of experts in use
        slab = 3 * H * I / 2 + 2 * (2 * _groups(H, group) * I + _groups(I, group) * H)
        return dict(bytes=active * slab + 4 * T * H + 8 * T * k, flops=6 * T * k * H * I)
    T, E, k, b = case["T"], case["E"], case["k"], 4 if case["dtype"] == "fp32" else 2
    return dict(bytes=T * E * b * (2 if case["grad"] else 1) + 4 * T * k + 4 * case["n_seq"] * E, flops=(8 if case["grad"] else 5) * T * E)


def exact(case, seed):
    """The definitions in 64 bits, expert by expert and sequence by sequence."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    F = torch.float64
    if st["op"] == "linear":
        K, N = st["codes"].shape
        y = torch.zeros(st["x"].shape[0], N, dtype=F, device="cuda")
        for g0 in range(0, K, st["group"]):
            part = st["x"][:, g0:g0 + st["group"]].to(F) @ (st["codes"][g0:g0 + st["group"]].to(F) - 8)
            y += part * st["scales"][g0 // st["group"]].to(F)
        return y
    if st["op"] == "experts":
        ids, H, I, group = st["ids"].cpu().numpy(), st["H"], st["I"], st["group"]
        gh, gi = _groups(H, group), _groups(I, group)
        e2s = st["e2s"].cpu().numpy()
        out = torch.zeros(ids.shape[0], H, dtype=F, device="cuda")
        for e in np.unique(ids):
            t, j = (torch.from_numpy(v).cuda() for v in np.nonzero(ids == e))
            c, s = st["codes"][int(e2s[e])].to(F) - 8, st["scales"][int(e2s[e])].to(F)
            n = H * I
            wide = lambda v, K: v.repeat_interleave(group, 0)[:K]  # noqa: E731
            wg = c[:n].view(H, I) * wide(s[:gh * I].view(gh, I), H)
            wu = c[n:2 * n].view(H, I) * wide(s[gh * I:2 * gh * I].view(gh, I), H)
            wd = c[2 * n:].view(I, H) * wide(s[2 * gh * I:].view(gi, H), I)
            xe = st["x"][t].to(F)
            a = xe @ wg
            out.index_add_(0, t, ((a * torch.sigmoid(a)) * (xe @ wu)) @ wd * st["w"][t, j].to(F)[:, None])
        return out
    logits, ids = st["logits"].to(F), st["ids"].cpu().numpy()
    T, E = logits.shape
    k = ids.shape[1]
    valid = np.ones(T, bool) if st["mask"] is None else st["mask"].cpu().numpy()
    starts = st["starts"].cpu().numpy()
    total = max(1, int(valid.sum()))
    loss, grad = 0.0, torch.zeros(T, E, dtype=F, device="cuda")
    counts = np.zeros((len(starts) - 1, E), np.int32)
    for s in range(len(starts) - 1):
        t = np.arange(starts[s], starts[s + 1])
        t = t[valid[t]]
        if not len(t):
            continue
        counts[s] = np.bincount(ids[t].reshape(-1), minlength=E)
        f = torch.from_numpy(counts[s] * (E / (k * len(t)))).cuda()
        i = torch.from_numpy(t).cuda()
        if st["sigmoid"]:
            a = torch.sigmoid(logits[i])
            p, jac = a / a.sum(1, keepdim=True), 1 - a
        else:
            p, jac = torch.softmax(logits[i], 1), 1.0
        d = p @ f
        loss += st["coef"] * float(d.sum()) / total
        grad[i] = st["coef"] / total * p * (f - d[:, None]) * jac
    return dict(loss=torch.tensor(loss, dtype=F), counts=counts, grad=grad if st["grad"] else None)
