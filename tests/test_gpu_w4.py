"""4-bit weights with group scales: packing, the linear layer, the grouped expert FFN, the routed experts.

Everything is compared with plain fp64 products of the unpacked weights (code - 8) * scale.

Tolerances.  Linear: the products of bf16 activations and 4-bit codes are exact, so an output's error comes from
its sums: at most K / 32 + 40 fp32 roundings on any path (16 inside an MMA, one per scaled block, the warps' and
parts' sums), each at most 2^-23 of the sum of |x w|.  A bf16 output adds half a unit in the last place, 2^-8 of
the value at most.  The expert FFN hands h to the down product with 16 (small batches) or 11 significant bits:
relative L2 errors of 2^-17 / 2^-12 and below in h and so in y, a factor two allowed on top; bf16 outputs are
off by up to 2^-8 / sqrt(3) / 1.2 = 1.9e-3 in relative L2 from their own rounding.
"""
import numpy as np
import pytest
import torch

from harness import configs as C
from tests._setup import rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"
RL2_Y_SMALL = 2.0 ** -16 + 1e-5
RL2_Y_LARGE = 2.0 ** -11
RL2_OUT_BF16 = 2.4e-3


def draw_w4(K, N, group, seed, lead=()):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, (*lead, K, N), generator=g, dtype=torch.uint8)
    scales = (torch.randn(*lead, -(-K // group), N, generator=g).mul(0.4).exp() * 0.01).to(torch.bfloat16)
    scales[..., 0, :: 7] *= -1  # scales carry a sign
    return codes, scales


def dequant(codes, scales, group):
    K = codes.shape[-2]
    return (codes.double() - 8) * scales.double().repeat_interleave(group, dim=-2)[..., :K, :]


def check_linear(y, x, w, out_dtype):
    want, mag = x.double() @ w, x.double().abs() @ w.abs()
    tol = (x.shape[1] / 32 + 40) * 2.0 ** -23 * mag
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp(min=1e-300)).max()):.2f} of the tolerance"


SHAPES = [(8, 1), (64, 16), (72, 17), (256, 33), (1416, 1001), (768, 2048), (2048, 130)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K,N", SHAPES)
def test_pack_holds_every_weight(K, N, group):
    """One-hot rows read the packed matrix back: every weight, bit for bit."""
    import expert_slot_cache_gb300 as M
    codes, scales = draw_w4(K, N, group, K + N)
    packed = M.w4_pack(codes.to(DEV), scales.to(DEV), group)
    assert packed.numel() == M.w4_bytes(K, N, group)
    want = dequant(codes, scales, group).float()
    rows = torch.arange(0, K, max(1, K // 61))
    x = torch.zeros(len(rows), K, dtype=torch.bfloat16)
    x[torch.arange(len(rows)), rows] = 1.0
    for part in range(0, len(rows), 16):
        op = M.W4Linear(packed, K, N, group, max_tokens=16, out_dtype=torch.float32)
        assert torch.equal(op.forward(x[part:part + 16].to(DEV)).cpu(), want[rows[part:part + 16]])


def quantize_plain(w, group):
    """The documented rule in fp32 (numpy): scale = bf16(m / -8) of the element furthest from zero."""
    K, N = w.shape
    q = np.zeros((K, N))
    w = w.float().numpy()
    for k0 in range(0, K, group):
        b = w[k0:k0 + group]
        hi, lo = np.maximum(b.max(0), 0), np.minimum(b.min(0), 0)
        m = np.where(hi > -lo, hi, lo).astype(np.float32)
        s = torch.from_numpy(m * np.float32(-0.125)).to(torch.bfloat16).float().numpy()
        with np.errstate(divide="ignore", invalid="ignore"):
            c = np.where(s != 0, np.clip(np.rint(b / s), -8, 7), 0)
        q[k0:k0 + group] = c * s.astype(np.float64)
    return q


@pytest.mark.parametrize("K,N,group", [(200, 40, 64), (256, 128, 128), (96, 19, 32)])
def test_quantize_follows_the_rule(K, N, group):
    import expert_slot_cache_gb300 as M
    g = torch.Generator().manual_seed(K)
    w = (torch.randn(K, N, generator=g) * 0.02).to(torch.bfloat16)
    w[: min(K, group), 3] = 0  # a group of zeros
    w[5, 4] = w[6, 4] = 0
    want = quantize_plain(w, group)
    packed = M.w4_quantize(w.to(DEV), group)
    op = M.W4Linear(packed, K, N, group, max_tokens=8, out_dtype=torch.float32)
    for k0 in range(0, K, 8):
        x = torch.zeros(8, K, dtype=torch.bfloat16)
        x[torch.arange(8), torch.arange(k0, k0 + 8)] = 1.0
        assert np.array_equal(op.forward(x.to(DEV)).cpu().numpy(), want[k0:k0 + 8].astype(np.float32))


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 31, 33, 65, 130, 300])
@pytest.mark.parametrize("K,N,group", [(2048, 256, 128), (1416, 1001, 32), (72, 17, 64), (4096, 48, 64)])
def test_linear(K, N, group, T, out_dtype):
    import expert_slot_cache_gb300 as M
    codes, scales = draw_w4(K, N, group, T)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T + 1)).to(torch.bfloat16)
    x[:, :: 97] *= 30
    op = M.W4Linear(M.w4_pack(codes.to(DEV), scales.to(DEV), group), K, N, group, max_tokens=T, out_dtype=out_dtype)
    y = op.forward(x.to(DEV))
    assert y.dtype == out_dtype and int(op.dev_status.item()) == 0
    check_linear(y, x, dequant(codes, scales, group), out_dtype)


@pytest.mark.parametrize("T", [3, 200])
def test_linear_strided_rows_and_wide_scales(T):
    """Rows of x and out inside wider tensors; neighbours stay as they were; NaN beside the rows is not read."""
    import expert_slot_cache_gb300 as M
    K, N, group = 264, 70, 64
    codes, scales = draw_w4(K, N, group, 5)
    scales[1] *= 2.0 ** -10  # far below the column's largest scale
    scales[2, ::2] = 0
    wide = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    wide[:, 8:8 + K] = x.to(DEV)
    out = torch.full((T, N + 5), 7.0, dtype=torch.float32, device=DEV)
    op = M.W4Linear(M.w4_pack(codes.to(DEV), scales.to(DEV), group), K, N, group, max_tokens=T, out_dtype=torch.float32)
    op.forward(wide[:, 8:8 + K], out=out[:, 2:2 + N])
    check_linear(out[:, 2:2 + N].contiguous(), x, dequant(codes, scales, group), torch.float32)
    assert bool((out[:, :2] == 7).all()) and bool((out[:, 2 + N:] == 7).all())


@pytest.mark.parametrize("T", [4, 256])
def test_linear_extreme_rows(T):
    """Rows of very large and very small values, of zeros, and rows with an infinity or a NaN beside sound ones."""
    import expert_slot_cache_gb300 as M
    K, N, group = 512, 96, 128
    codes, scales = draw_w4(K, N, group, 9)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[0] = 0
    x[1] *= 2.0 ** 90
    x[2] *= 2.0 ** -90
    op = M.W4Linear(M.w4_pack(codes.to(DEV), scales.to(DEV), group), K, N, group, max_tokens=T, out_dtype=torch.float32)
    w = dequant(codes, scales, group)
    check_linear(op.forward(x.to(DEV)), x, w, torch.float32)
    x[3, 5] = float("nan")
    x[1, 7] = float("inf")
    y = op.forward(x.to(DEV)).cpu()
    assert bool(y[3].isnan().all())
    assert not bool(y[1].isfinite().any())
    keep = [0, 2] + list(range(4, T))
    check_linear(y[keep], x[keep], w, torch.float32)


def test_linear_is_the_same_on_any_stream_and_run():
    import expert_slot_cache_gb300 as M
    K, N, group = 2048, 2048, 128
    codes, scales = draw_w4(K, N, group, 1)
    packed = M.w4_pack(codes.to(DEV), scales.to(DEV), group)
    for T in (1, 64, 512):
        x = torch.randn(T, K, device=DEV).to(torch.bfloat16)
        op = M.W4Linear(packed, K, N, group, max_tokens=T)
        first = op.forward(x)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            others = [op.forward(x) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(first, o) for o in others)


# ---------------------------------------------------------------------------
# Experts
# ---------------------------------------------------------------------------

def draw_experts(H, I, E, group, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 16, (E, 3 * H * I), generator=g, dtype=torch.uint8, device=DEV)
    n = 2 * -(-H // group) * I + -(-I // group) * H
    scales = (torch.randn(E, n, generator=g, device=DEV).mul(0.3).exp() * 0.006).to(torch.bfloat16)
    return codes, scales


def expert_mats(codes, scales, H, I, group):
    gh, gi = -(-H // group), -(-I // group)
    c, s = codes.split([H * I, H * I, I * H]), scales.split([gh * I, gh * I, gi * H])
    return [dequant(a.view(K, N), b.view(-1, N), group) for a, b, (K, N) in zip(c, s, [(H, I), (H, I), (I, H)])]


def ffn_plain(x, codes, scales, H, I, group):
    wg, wu, wd = expert_mats(codes, scales, H, I, group)
    a = x.double() @ wg
    return (a * torch.sigmoid(a) * (x.double() @ wu)) @ wd


def experts_plain(x, ids, w, codes, scales, H, I, group, skip=()):
    out = torch.zeros(x.shape[0], H, dtype=torch.float64, device=DEV)
    for e in torch.unique(ids).tolist():
        if e in skip or not 0 <= e < codes.shape[0]:
            continue
        t, j = torch.nonzero(ids == e, as_tuple=True)
        out.index_add_(0, t, ffn_plain(x[t], codes[e], scales[e], H, I, group) * w[t, j].double()[:, None])
    return out


def draw_routing(T, E, k, seed, skew=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = torch.randn(T, E, generator=g, device=DEV) - skew * torch.arange(E, device=DEV).log1p()
    top, ids = torch.topk(logits, k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, 1)


EXPERT_CASES = [
    ("tiny_T1", 256, 128, 16, 2, 1, 128, 0.0),
    ("tiny_T5_g32", 256, 128, 16, 2, 5, 32, 0.0),
    ("odd_T3", 320, 96, 11, 3, 3, 64, 0.0),
    ("odd_T40", 448, 416, 13, 5, 40, 128, 0.5),
    ("one_expert_T70", 128, 64, 1, 1, 70, 64, 0.0),
    ("qwen_T1", 2048, 768, 128, 8, 1, 128, 0.0),
    ("qwen_T8", 2048, 768, 128, 8, 8, 64, 0.3),
    ("qwen_T64", 2048, 768, 128, 8, 64, 128, 0.6),
    ("flash_T16", 2048, 512, 512, 10, 16, 64, 0.0),
    ("stack_T32", 2048, 512, 288, 8, 32, 32, 0.0),
    ("tiny_T700", 256, 128, 16, 2, 700, 64, 0.8),
    ("odd_T900", 320, 160, 9, 4, 900, 32, 1.0),
    ("qwen_T1200", 2048, 768, 32, 8, 1200, 128, 0.8),
]


@pytest.mark.parametrize("name,H,I,E,k,T,group,skew", EXPERT_CASES, ids=[c[0] for c in EXPERT_CASES])
def test_experts(name, H, I, E, k, T, group, skew):
    import expert_slot_cache_gb300 as M
    codes, scales = draw_experts(H, I, E, group, T)
    perm = torch.randperm(E, generator=torch.Generator().manual_seed(T)).to(DEV)
    pool = M.w4_pack_slabs(codes[perm].contiguous(), scales[perm].contiguous(), H, I, group)
    e2s = torch.empty(E, dtype=torch.int32, device=DEV)
    e2s[perm] = torch.arange(E, dtype=torch.int32, device=DEV)
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T + 7), device=DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, E, k, T, skew)
    op = M.W4Experts(pool, H, I, k, E, group, e2s=e2s, max_tokens=T)
    out = op.forward(x, ids, w)
    assert int(op.dev_status.item()) == 0
    want = experts_plain(x, ids, w, codes, scales, H, I, group)
    r = rel_l2(out.double().cpu(), want.cpu())
    assert r <= RL2_OUT_BF16, r
    worst = ((out.double() - want).norm(dim=1) / want.norm(dim=1)).max()  # no token on its own is far off
    assert float(worst) <= 2 * RL2_OUT_BF16, float(worst)
    assert torch.equal(out, op.forward(x, ids, w))
    # the list form: fp32 rows
    g = M.permute(ids, E)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = M.expert_ffn_w4(x, k, I, E, group, g.offset, g.rows, g.act_e, g.n_act, E, pool, e2s=e2s, dev_status=st)
    assert int(st.item()) == 0
    rows = g.rows.long()
    flat = ids.reshape(-1).long()
    bad = 0.0
    for e in torch.unique(flat).tolist()[:24]:
        p = torch.nonzero(flat[rows] == e).reshape(-1)
        wy = ffn_plain(x[rows[p] // k], codes[e], scales[e], H, I, group)
        bad = max(bad, rel_l2(y[p].cpu(), wy.cpu()))
    assert bad <= (RL2_Y_SMALL if T * k <= 128 else RL2_Y_LARGE), bad


@pytest.mark.parametrize("T", [1, 6, 300])
def test_experts_bad_ids_and_missing_slots(T):
    """Out-of-range ids and experts without a slot add nothing and are flagged; the same expert may come twice."""
    import expert_slot_cache_gb300 as M
    H, I, E, k, group = 256, 128, 16, 3, 64
    codes, scales = draw_experts(H, I, E, group, 3)
    S = 12
    pool = M.w4_pack_slabs(codes[:S].contiguous(), scales[:S].contiguous(), H, I, group)
    e2s = torch.full((E,), -1, dtype=torch.int32, device=DEV)
    e2s[:S] = torch.arange(S, dtype=torch.int32, device=DEV)
    e2s[13] = 4000  # a slot outside the pool
    x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, S, k, 5)
    ids[:, 1] = ids[:, 0]  # one expert twice
    op = M.W4Experts(pool, H, I, k, E, group, e2s=e2s, max_tokens=T)
    want = experts_plain(x, ids, w, codes, scales, H, I, group)
    assert rel_l2(op.forward(x, ids, w).double().cpu(), want.cpu()) <= RL2_OUT_BF16
    assert int(op.dev_status.item()) == 0
    for bad, code in ((-1, 1), (E, 1), (2 ** 30, 1), (12, 2), (13, 2)):
        b = ids.clone()
        b[0, 2] = bad
        want = experts_plain(x, b, w, codes, scales, H, I, group, skip=(12, 13))
        out = op.forward(x, b, w)
        assert int(op.dev_status.item()) == code, bad
        op.dev_status.zero_()
        assert rel_l2(out.double().cpu(), want.cpu()) <= RL2_OUT_BF16, bad
    b = torch.full_like(ids, -1)  # nothing routed at all
    assert not bool(op.forward(x, b, w).any())


@pytest.mark.parametrize("mode,T,S,sched", [(C.MODE_RESIDENT, 5, 16, 0), (C.MODE_GATHER, 3, 8, C.SCHED_CHUNKS),
                                            (C.MODE_GATHER, 20, 8, C.SCHED_CHUNKS),
                                            (C.MODE_GATHER, 20, 8, C.SCHED_WAVES)],
                         ids=["resident", "gather", "gather_chunks", "gather_waves"])
def test_layer_with_4bit_slabs(mode, T, S, sched):
    """The whole layer over 4-bit slabs: slots, misses and the gather move packed slabs; the output is the experts'."""
    import expert_slot_cache_gb300 as M
    cfg = C.TINY.with_(T=T, S=S, mode=mode)
    H, I, E, k, group = cfg.H, cfg.I, cfg.E, cfg.k, 64
    slabs = torch.empty(E, cfg.slab_elems, dtype=torch.bfloat16, device=DEV)
    C.draw_slabs(cfg, DEV, out=slabs)
    slabs *= 4
    packed = M.w4_quantize_slabs(slabs, H, I, group)
    wr = C.draw_router(cfg, DEV)
    state = host = None
    pool = packed
    if mode == C.MODE_GATHER:
        s2e = C.initial_residency(cfg)
        host = torch.empty(packed.shape, dtype=torch.uint8, pin_memory=True)
        host.copy_(packed)
        pool = packed[torch.from_numpy(s2e.astype(np.int64)).to(DEV)].contiguous()
        state = M.CacheState.from_slots(s2e, E)
    layer = M.SlotCachedMoELayer(wr, pool, k, I, mode, C.POLICY_LRU, host_slabs=host, state=state, max_tokens=T,
                                 quant=2, quant_group=group, schedule=sched)
    q = [torch.from_numpy(np.concatenate([quantize_plain(m, group).reshape(-1) for m in
                                          (s[:H * I].view(H, I), s[H * I:2 * H * I].view(H, I), s[2 * H * I:].view(I, H))]))
         for s in slabs.cpu()]
    for step in range(3):
        x = C.draw_x(cfg, DEV, step=step)
        res = layer.forward(x)
        torch.cuda.synchronize()
        want = torch.zeros(T, H, dtype=torch.float64)
        xd = x.double().cpu()
        for t in range(T):
            for j in range(k):
                e = int(res["ids"][t, j])
                wg, wu, wd = q[e][:H * I].view(H, I), q[e][H * I:2 * H * I].view(H, I), q[e][2 * H * I:].view(I, H)
                a = xd[t] @ wg
                want[t] += float(res["w"][t, j]) * ((a * torch.sigmoid(a) * (xd[t] @ wu)) @ wd)
        assert rel_l2(res["out"].double().cpu(), want) <= RL2_OUT_BF16, step
    assert int(layer.dev_status.item()) == 0
    if mode == C.MODE_GATHER:
        for s, e in enumerate(state.s2e.cpu().tolist()):
            assert torch.equal(pool[s].cpu(), host[e])
