"""The 4-bit operators at larger sizes: the linear layer on the large tensor-core tiles (from 17 rows, by rows x
weights), and many experts of few rows.

Compared with fp64 products of the unpacked weights, with the tolerance of the small sizes: (K / 32 + 40) fp32
roundings of 2^-23 of the sum of |x w| at most (parts of the inputs that are summed apart add one rounding each,
of the 40), and half a unit in the last place of a bf16 output.
"""
import pytest
import torch

from harness import configs as C
from tests._setup import rel_l2
from tests.test_gpu_w4 import (RL2_OUT_BF16, check_linear, dequant, draw_experts, draw_routing, draw_w4,
                               experts_plain)
from tests import test_gpu_w4 as small

pytestmark = pytest.mark.gpu
DEV = "cuda"

# K, N, group, T: many parts of few columns; ragged columns; one, two and several row tiles; an odd number of
# stages, and a last stage that is mostly past K; one row more than a pass of the small kernel
CASES = [(16392, 520, 64, 40), (4104, 4097, 32, 33), (8200, 4160, 128, 17), (2064, 3000, 64, 300),
         (1032, 1001, 128, 600), (136, 100003, 32, 65), (520, 2049, 128, 513), (4096, 2112, 64, 257)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K,N,group,T", CASES)
def test_linear(K, N, group, T, out_dtype):
    import expert_slot_cache_gb300 as M
    codes, scales = draw_w4(K, N, group, T)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T + 1)).to(torch.bfloat16)
    x[:, :: 97] *= 30
    op = M.W4Linear(M.w4_pack(codes.to(DEV), scales.to(DEV), group), K, N, group, max_tokens=T, out_dtype=out_dtype)
    y = op.forward(x.to(DEV))
    assert int(op.dev_status.item()) == 0
    check_linear(y, x, dequant(codes, scales, group), out_dtype)


@pytest.mark.parametrize("K,N,T", [(4104, 1100, 130), (2056, 5000, 70)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_strided_rows(K, N, T, out_dtype):
    """Rows of x and out inside wider tensors, fewer of them than the operator was made for."""
    import expert_slot_cache_gb300 as M
    codes, scales = draw_w4(K, N, 64, 5)
    wide = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    wide[:, 8:8 + K] = x.to(DEV)
    out = torch.full((T, N + 5), 7.0, dtype=out_dtype, device=DEV)
    op = M.W4Linear(M.w4_pack(codes.to(DEV), scales.to(DEV), 64), K, N, 64, max_tokens=3000, out_dtype=out_dtype)
    op.forward(wide[:, 8:8 + K], out=out[:, 2:2 + N])
    check_linear(out[:, 2:2 + N].contiguous(), x, dequant(codes, scales, 64), out_dtype)
    assert bool((out[:, :2] == 7).all()) and bool((out[:, 2 + N:] == 7).all())


def test_extreme_rows():
    """Rows of very large and very small values and of zeros; infinities and NaN stay in their rows."""
    import expert_slot_cache_gb300 as M
    T, K, N, group = 90, 4096, 1536, 128
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
    assert bool(y[3].isnan().all()) and not bool(y[1].isfinite().any())
    keep = [0, 2] + list(range(4, T))
    check_linear(y[keep], x[keep], w, torch.float32)


def test_same_result_every_time():
    import expert_slot_cache_gb300 as M
    T, K, N, group = 200, 4096, 1024, 64
    codes, scales = draw_w4(K, N, group, 1)
    op = M.W4Linear(M.w4_pack(codes.to(DEV), scales.to(DEV), group), K, N, group, max_tokens=T)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    want = op.forward(x).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            assert torch.equal(op.forward(x), want)


# more routing slots than the stream kernels group themselves, few of them for each expert
MANY_EXPERTS = [("qwen_T100", 2048, 768, 128, 8, 100, 128, 0.5), ("many_T600", 256, 128, 300, 4, 600, 64, 0.3),
                ("most_T1100", 128, 64, 1024, 9, 1100, 32, 0.1), ("edge_T64", 448, 96, 100, 8, 64, 64, 0.0),
                ("edge_T65", 448, 96, 100, 8, 65, 64, 0.0)]


@pytest.mark.parametrize("name,H,I,E,k,T,group,skew", MANY_EXPERTS, ids=[c[0] for c in MANY_EXPERTS])
def test_experts_of_few_rows(name, H, I, E, k, T, group, skew):
    small.test_experts(name, H, I, E, k, T, group, skew)


def test_experts_missing_slots_in_groups():
    import expert_slot_cache_gb300 as M
    H, I, E, k, group, S, T = 128, 64, 100, 6, 64, 90, 160
    codes, scales = draw_experts(H, I, E, group, 3)
    pool = M.w4_pack_slabs(codes[:S].contiguous(), scales[:S].contiguous(), H, I, group)
    e2s = torch.full((E,), -1, dtype=torch.int32, device=DEV)
    e2s[:S] = torch.arange(S, dtype=torch.int32, device=DEV)
    x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, S, k, 5)
    ids[3, 2], ids[5, 0], ids[7, 1] = -1, E, 95  # not experts; an expert without a slot
    op = M.W4Experts(pool, H, I, k, E, group, e2s=e2s, max_tokens=T)
    want = experts_plain(x, ids, w, codes, scales, H, I, group, skip=range(S, E))
    assert rel_l2(op.forward(x, ids, w).double().cpu(), want.cpu()) <= RL2_OUT_BF16
    assert int(op.dev_status.item()) != 0


def test_experts_any_batch_up_to_the_largest():
    """An operator made for many tokens takes every smaller batch, whichever way it is computed."""
    import expert_slot_cache_gb300 as M
    H, I, E, k, group = 128, 256, 20, 4, 64
    codes, scales = draw_experts(H, I, E, group, 8)
    pool = M.w4_pack_slabs(codes, scales, H, I, group)
    for most in (50, 51, 600):
        op = M.W4Experts(pool, H, I, k, E, group, max_tokens=most)
        for T in sorted({1, 4, 5, 31, 32, 33, 49, 50, most}):
            x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
            ids, w = draw_routing(T, E, k, T)
            want = experts_plain(x, ids, w, codes, scales, H, I, group)
            assert rel_l2(op.forward(x, ids, w).double().cpu(), want.cpu()) <= RL2_OUT_BF16, (most, T)


@pytest.mark.parametrize("H,I,E,k,T,group", [(2048, 768, 128, 8, 717, 32), (1024, 256, 64, 8, 500, 128)])
def test_experts_same_result_every_time(H, I, E, k, T, group):
    """Weights read from memory and from the caches, in turn: copies that land in any order."""
    import expert_slot_cache_gb300 as M
    codes, scales = draw_experts(H, I, E, group, T)
    pool = M.w4_pack_slabs(codes, scales, H, I, group)
    x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, E, k, T, 0.4)
    op = M.W4Experts(pool, H, I, k, E, group, max_tokens=T)
    want = op.forward(x, ids, w).clone()
    assert rel_l2(want.double().cpu(), experts_plain(x, ids, w, codes, scales, H, I, group).cpu()) <= RL2_OUT_BF16
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    same = torch.ones((), dtype=torch.bool, device=DEV)
    for i in range(400):
        if i % 4 == 0:
            flush.fill_(i % 256)
        same &= (op.forward(x, ids, w) == want).all()
    assert bool(same) and int(op.dev_status.item()) == 0


@pytest.mark.parametrize("mode,T,S,sched", [(C.MODE_RESIDENT, 120, 16, 0), (C.MODE_GATHER, 120, 8, C.SCHED_CHUNKS),
                                            (C.MODE_GATHER, 120, 8, C.SCHED_WAVES)],
                         ids=["resident", "gather_chunks", "gather_waves"])
def test_layer_with_4bit_slabs(mode, T, S, sched):
    """The layer's larger steps: experts of many rows, hits and misses as lists of their own."""
    small.test_layer_with_4bit_slabs(mode, T, S, sched)
