"""A 4-bit matrix of more columns than 128 times a grid's y or z."""
import pytest
import torch

from tests.test_gpu_w4 import dequant

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("quantized", [False, True])
def test_columns_beyond_eight_million(quantized):
    """Products of one-hot rows read weights back; K = 16: every result is exact."""
    import expert_slot_cache_gb300 as M
    K, N, group = 16, 65535 * 128 + 133, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    codes = torch.randint(0, 16, (K, N), generator=g, device=DEV, dtype=torch.uint8)
    scales = (torch.rand(1, N, generator=g, device=DEV) + 0.5).to(torch.bfloat16)
    if quantized:  # code 0 in every column: the rule gives codes and scales back
        codes[3] = 0
        packed = M.w4_quantize(dequant(codes, scales, group).to(torch.bfloat16), group)
    else:
        packed = M.w4_pack(codes, scales, group)
    assert packed.numel() == M.w4_bytes(K, N, group)
    op = M.W4Linear(packed, K, N, group, max_tokens=3, out_dtype=torch.float32)
    for rows in ((0, 3, 7), (8, 15, 2)):
        x = torch.zeros(3, K, dtype=torch.bfloat16, device=DEV)
        x[torch.arange(3), torch.tensor(rows)] = 1.0
        want = (codes[list(rows)].float() - 8) * scales.float()
        if quantized:
            want = want.to(torch.bfloat16).float()
            assert bool(((op.forward(x) - want).abs() <= 0.5 * scales.float()).all())
        else:
            assert torch.equal(op.forward(x), want)
