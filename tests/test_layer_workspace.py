"""The layer's workspace: what the bf16 and W8A8 paths need, and no more on behalf of 4-bit slabs, which take their
buffers from the same place."""
import pytest
import torch


@pytest.fixture(scope="module")
def b():
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as binding
    return binding


# above 4096 routing slots: h fp32, y fp32, the grouped rows and h in bf16, the logits, the router's and the permute's
# scratch, and the lists of rows and experts
@pytest.mark.parametrize("T,H,E,k,I", [(4096, 2048, 128, 8, 768), (600, 2048, 512, 10, 512), (5000, 256, 16, 2, 128)])
def test_size_of_large_steps(b, T, H, E, k, I):
    n = T * k
    parts = 4 * n * I + 4 * n * H + 2 * n * H + 2 * n * I + 4 * T * E
    scratch = int(b._route_scratch(T, H, E)) + int(b._permute_scratch(n, E))
    # (a step in chunks of up to 4096 slots needs a chunk's buffers and the whole step's logits)
    most = max(parts + scratch + 16 * n + 64 * E + (1 << 16),
               b.layer_workspace_bytes(4096 // k, H, E, k, I, E) + 4 * T * E + scratch + (1 << 16))
    assert b.layer_workspace_bytes(T, H, E, k, I, E) <= most


SHAPES = [(256, 96, 16, 8, 21), (320, 32, 8, 3, 43), (256, 128, 24, 8, 511), (256, 96, 24, 8, 513), (64, 32, 40, 9, 900)]


def test_every_form_fits(b):
    """4-bit buffers within 4nI of h and the room for bf16 rows and h (kept by every size)."""
    for n in list(range(1, 700)) + [4095, 4096, 4097, 10240, 1 << 20]:
        for H, I in ((64, 32), (256, 96), (2048, 768), (7168, 2048), (128, 4096)):
            assert int(b._ffn_w4_ws(n, H, 1, I)) <= 4 * n * I + 2 * n * H + 2 * n * I + 768, (n, H, I)


@pytest.mark.gpu
@pytest.mark.parametrize("H,I,E,k,T", SHAPES)
def test_layer_over_4bit_slabs_stays_in_its_workspace(b, H, I, E, k, T):
    """Steps of every path (streams, large tiles; below and above 4096 slots) in a workspace of exactly the stated size."""
    from tests._setup import rel_l2
    from tests.test_gpu_w4 import RL2_OUT_BF16, draw_experts, experts_plain
    M, dev, group = b, "cuda", 64
    codes, scales = draw_experts(H, I, E, group, T)
    wr = torch.randn(H, E, generator=torch.Generator().manual_seed(1)).mul(H ** -0.5).to(torch.bfloat16).to(dev)
    layer = M.SlotCachedMoELayer(wr, M.w4_pack_slabs(codes, scales, H, I, group), k, I, M.MODE_RESIDENT, max_tokens=T,
                                 quant=2, quant_group=group)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).to(dev)
    for t in sorted({1, 5, T // 3 + 1, T}):
        size = M.layer_workspace_bytes(t, H, E, k, I, E)
        room = torch.zeros(size + 4096, dtype=torch.uint8, device=dev)
        room[size:] = 171
        layer.workspace = room[:size]
        r = layer.forward(x[:t])
        want = experts_plain(x[:t], r["ids"], r["w"], codes, scales, H, I, group)
        assert rel_l2(r["out"].double().cpu(), want.cpu()) <= RL2_OUT_BF16, t
        assert int(layer.dev_status.item()) == 0 and bool((room[size:] == 171).all()), t


def test_a_workspace_is_enough_for_fewer_tokens(b):
    for H, E, k, I in ((256, 24, 8, 96), (64, 40, 9, 32), (256, 16, 2, 128), (2048, 128, 8, 768)):
        sizes = [b.layer_workspace_bytes(T, H, E, k, I, E) for T in (1, 2, 7, 60, 100, 172, 300, 455, 512, 513, 900, 2048, 2049, 5000)]
        assert sizes == sorted(sizes), (H, E, k, I)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [0, 2])
@pytest.mark.parametrize("H,I,E,k,T", SHAPES)
def test_a_layer_takes_every_smaller_step(b, H, I, E, k, T, quant):
    """Steps of 1 to max_tokens tokens of one layer (split sums below 4096 slots, none above)."""
    from tests._setup import rel_l2
    from tests.test_gpu_w4 import RL2_OUT_BF16, draw_experts, expert_mats, experts_plain
    M, dev, group = b, "cuda", 64
    codes, scales = draw_experts(H, I, E, group, T)
    slabs = (M.w4_pack_slabs(codes, scales, H, I, group) if quant else
             torch.stack([torch.cat([m.reshape(-1) for m in expert_mats(codes[e], scales[e], H, I, group)]) for e in range(E)]).to(torch.bfloat16))
    wr = torch.randn(H, E, generator=torch.Generator().manual_seed(1)).mul(H ** -0.5).to(torch.bfloat16).to(dev)
    layer = M.SlotCachedMoELayer(wr, slabs, k, I, M.MODE_RESIDENT, max_tokens=T, quant=quant, quant_group=group)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).to(dev)
    for t in sorted({1, 5, T // 3 + 1, T}):
        r = layer.forward(x[:t])
        want = experts_plain(x[:t], r["ids"], r["w"], codes, scales, H, I, group)
        # bf16 slabs: the weights' own rounding and that of h and y to bf16, 2^-8 / sqrt(12) / 0.69 each at most
        assert rel_l2(r["out"].double().cpu(), want.cpu()) <= (RL2_OUT_BF16 if quant else 4 * RL2_OUT_BF16), t
    assert int(layer.dev_status.item()) == 0
