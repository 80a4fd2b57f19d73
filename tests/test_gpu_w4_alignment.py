"""The routed 4-bit experts into an output that is 8-byte but not 16-byte aligned, on every path."""
import pytest
import torch

from tests._setup import rel_l2
from tests.test_gpu_w4 import RL2_OUT_BF16, draw_experts, draw_routing, experts_plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [1, 30, 70, 400])  # own groups, given groups, large tiles (10 rows of an expert and more)
def test_out_on_eight_bytes(T):
    import expert_slot_cache_gb300 as M
    H, I, E, k, group = 320, 96, 12, 4, 64
    codes, scales = draw_experts(H, I, E, group, 2)
    op = M.W4Experts(M.w4_pack_slabs(codes, scales, H, I, group), H, I, k, E, group, max_tokens=T)
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, E, k, T)
    buf = torch.full((T * H + 8,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[4:4 + T * H].view(T, H)
    assert out.data_ptr() % 16 == 8
    op.forward(x, ids, w, out=out)
    assert torch.equal(out, op.forward(x, ids, w))
    assert rel_l2(out.double().cpu(), experts_plain(x, ids, w, codes, scales, H, I, group).cpu()) <= RL2_OUT_BF16
    assert bool((buf[:4] == 7).all()) and bool((buf[4 + T * H:] == 7).all())
