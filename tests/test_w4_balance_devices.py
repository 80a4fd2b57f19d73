"""The 4-bit and balance entry points refuse tensors that are not on the device that the call runs on (no GPU: the
refusal comes before any CUDA call; the "meta" device stands for another one)."""
import pytest
import torch

Z = torch.zeros


@pytest.fixture(scope="module")
def b():
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as binding
    return binding


def test_host_tensors(b):
    u8, bf, i32 = torch.uint8, torch.bfloat16, torch.int32
    lin = b.W4Linear(Z(b.w4_bytes(64, 16, 64), dtype=u8), 64, 16, 64, max_tokens=2)
    ex = b.W4Experts(Z(16, b.w4_slab_bytes(256, 128, 64), dtype=u8), 256, 128, 2, 16, 64, max_tokens=2)
    n = 3 * 256 * 128
    calls = [lambda: b.w4_pack(Z(64, 16, dtype=u8), Z(1, 16, dtype=bf), 64), lambda: b.w4_quantize(Z(64, 16, dtype=bf), 64),
             lambda: b.w4_pack_slabs(Z(2, n, dtype=u8), Z(2, 2 * 4 * 128 + 2 * 256, dtype=bf), 256, 128, 64),
             lambda: b.w4_quantize_slabs(Z(2, n, dtype=bf), 256, 128, 64), lambda: lin.forward(Z(2, 64, dtype=bf)),
             lambda: ex.forward(Z(2, 256, dtype=bf), Z(2, 2, dtype=i32), Z(2, 2)),
             lambda: b.expert_ffn_w4(Z(2, 256, dtype=bf), 2, 128, 16, 64, *[Z(17, dtype=i32)] * 4, 16, ex.pool),
             lambda: b.balance_loss(Z(4, 8), Z(4, 2, dtype=i32), 0.1)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_tensors_elsewhere(b):
    there = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="seq_start: on cpu, the call runs on cuda:0"):
        b._on(there, ids=None, seq_start=Z(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="x: on meta"):
        b._on(there, x=torch.zeros(3, device="meta"))


@pytest.mark.gpu
def test_host_indices_beside_device_tensors(b):
    """Refused on the host: none of these pointers reaches a kernel."""
    M, dev = b, "cuda"
    logits, ids = torch.randn(8, 16, device=dev), Z(8, 2, dtype=torch.int32)
    starts, mask = torch.tensor([0, 8], dtype=torch.int32), torch.ones(8, dtype=torch.bool)
    with pytest.raises(ValueError, match="ids"):
        M.balance_loss(logits, ids, 0.1)
    ids = ids.to(dev)
    with pytest.raises(ValueError, match="seq_start"):
        M.balance_loss(logits, ids, 0.1, starts)
    with pytest.raises(ValueError, match="token_mask"):
        M.balance_loss(logits, ids, 0.1, starts.to(dev), mask)
    with pytest.raises(ValueError, match="grad_loss"):
        M.balance_loss(logits, ids, 0.1, starts.to(dev), mask.to(dev), with_grad=True, grad_loss=torch.ones(1))
    assert M.balance_loss(logits, ids, 0.1, starts.to(dev), mask.to(dev)).loss.isfinite()
    pool = Z(16, M.w4_slab_bytes(256, 128, 64), dtype=torch.uint8, device=dev)
    ex = M.W4Experts(pool, 256, 128, 2, 16, 64, max_tokens=8)
    x = Z(8, 256, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError, match="ids"):
        ex.forward(x, ids.cpu(), Z(8, 2, device=dev))
    with pytest.raises(ValueError, match="w: on cpu"):
        ex.forward(x, ids, Z(8, 2))
    lin = M.W4Linear(Z(M.w4_bytes(256, 16, 64), dtype=torch.uint8, device=dev), 256, 16, 64, max_tokens=8)
    with pytest.raises(ValueError, match="x: on cpu"):
        lin.forward(x.cpu())
    with pytest.raises(ValueError, match="out: on cpu"):
        lin.forward(x, out=Z(8, 16, dtype=torch.bfloat16))
