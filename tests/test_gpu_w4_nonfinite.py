"""The routed 4-bit experts beside weights and scales that are not finite."""
import pytest
import torch

from tests._setup import rel_l2
from tests.test_gpu_w4 import RL2_OUT_BF16, draw_experts, draw_routing, experts_plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("weight", [float("inf"), float("nan")])
@pytest.mark.parametrize("T", [1, 9, 60, 300])  # the kernels' own groups, given groups, large tiles
def test_missing_experts_add_nothing_whatever_their_weight(T, weight):
    import expert_slot_cache_gb300 as M
    H, I, E, k, group, S = 128, 64, 60, 9, 64, 50
    codes, scales = draw_experts(H, I, E, group, 3)
    pool = M.w4_pack_slabs(codes[:S].contiguous(), scales[:S].contiguous(), H, I, group)
    e2s = torch.full((E,), -1, dtype=torch.int32, device=DEV)
    e2s[:S] = torch.arange(S, dtype=torch.int32, device=DEV)
    e2s[E - 1] = S  # outside the pool
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, S, k, 5)
    for t, j, e in ((0, 2, E - 2), (T // 2, 3, E - 1), (T - 1, 1, -1), (T - 1, 0, E)):
        ids[t, j], w[t, j] = e, weight
    op = M.W4Experts(pool, H, I, k, E, group, e2s=e2s, max_tokens=T)
    want = experts_plain(x, ids, w, codes, scales, H, I, group, skip=range(S, E))
    assert bool(want.isfinite().all())
    assert rel_l2(op.forward(x, ids, w).double().cpu(), want.cpu()) <= RL2_OUT_BF16
    assert int(op.dev_status.item()) != 0


@pytest.mark.parametrize("T", [1, 60])
def test_ids_past_the_experts_add_nothing_in_a_larger_pool(T):
    import expert_slot_cache_gb300 as M
    H, I, E, k, group, S = 128, 64, 60, 9, 64, 70
    codes, scales = draw_experts(H, I, S, group, 3)
    pool = M.w4_pack_slabs(codes, scales, H, I, group)
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, E, k, 5)
    ids[0, 2], w[0, 2] = E + 3, float("inf")
    op = M.W4Experts(pool, H, I, k, E, group, max_tokens=T)
    want = experts_plain(x, ids, w, codes[:E], scales[:E], H, I, group)
    assert bool(want.isfinite().all())
    assert rel_l2(op.forward(x, ids, w).double().cpu(), want.cpu()) <= RL2_OUT_BF16


@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
@pytest.mark.parametrize("T", [3, 200])
def test_a_column_without_finite_values_leaves_the_others(T, scale):
    """One output column of every expert has a scale that is not finite; the others are large."""
    import expert_slot_cache_gb300 as M
    H, I, E, k, group = 128, 64, 6, 3, 64
    codes, scales = draw_experts(H, I, E, group, 3)
    down = scales[:, 2 * (H // group) * I:].view(E, I // group, H)
    down *= 2.0 ** 24
    down[:, 0, 5] = scale
    op = M.W4Experts(M.w4_pack_slabs(codes, scales, H, I, group), H, I, k, E, group, max_tokens=T)
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, E, k, 5)
    out, want = op.forward(x, ids, w).double().cpu(), experts_plain(x, ids, w, codes, scales, H, I, group).cpu()
    others = [n for n in range(H) if n != 5]
    assert not bool(out[:, 5].isfinite().any()) and bool(want[:, others].isfinite().all())
    assert rel_l2(out[:, others], want[:, others]) <= RL2_OUT_BF16


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_quantising_does_not_hide_values_that_are_not_finite(value):
    """A weight without a finite value: its column gives none where its group is met, other columns and groups are as before."""
    import expert_slot_cache_gb300 as M
    K, N, group = 192, 40, 64
    w = (torch.randn(K, N, generator=torch.Generator().manual_seed(1)) * 0.02).to(torch.bfloat16).to(DEV)
    op = lambda w: M.W4Linear(M.w4_quantize(w, group), K, N, group, max_tokens=2, out_dtype=torch.float32)  # noqa: E731
    x = torch.randn(2, K, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    want = op(w).forward(x)
    w[70, 7] = value
    y = op(w).forward(x)
    others = [n for n in range(N) if n != 7]
    assert torch.equal(y[:, others], want[:, others])
    assert not bool(y[:, 7].isfinite().any())
