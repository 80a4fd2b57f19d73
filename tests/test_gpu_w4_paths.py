"""The 4-bit operators by path and as a program runs them: rows by the path that the sizes choose, graphs, streams,
stacks of layers, larger layers.

The list form's tolerance goes by the path: h reaches the down product with 16 bits where T k <= 128 or T k < 10 E (2^-17
and below, a factor two on top, 1e-5 for the fp32 sums), with 11 bits elsewhere (2^-12 and the factor two).
"""
import numpy as np
import pytest
import torch

from harness import configs as C
from tests._setup import rel_l2
from tests.test_gpu_w4 import (EXPERT_CASES, RL2_OUT_BF16, RL2_Y_LARGE, RL2_Y_SMALL, draw_experts, draw_routing, draw_w4,
                               experts_plain, ffn_plain)
from tests.test_gpu_w4_large import MANY_EXPERTS

pytestmark = pytest.mark.gpu
DEV = "cuda"

# 10 to 128 rows of an expert
MORE = [("rows12", 448, 160, 24, 6, 50, 64, 0.0), ("rows30", 1024, 96, 8, 4, 60, 32, 0.3), ("rows60", 256, 512, 16, 3, 320, 128, 0.0),
        ("rows100", 320, 288, 10, 5, 200, 64, 0.2)]
CASES = EXPERT_CASES + MANY_EXPERTS + MORE


@pytest.mark.parametrize("name,H,I,E,k,T,group,skew", CASES, ids=[c[0] for c in CASES])
def test_rows_of_lists_by_path(name, H, I, E, k, T, group, skew):
    import expert_slot_cache_gb300 as M
    codes, scales = draw_experts(H, I, E, group, T + 1)
    pool = M.w4_pack_slabs(codes, scales, H, I, group)
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T + 8), device=DEV).to(torch.bfloat16)
    ids, _ = draw_routing(T, E, k, T + 1, skew)
    g = M.permute(ids, E)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = M.expert_ffn_w4(x, k, I, E, group, g.offset, g.rows, g.act_e, g.n_act, E, pool, dev_status=st)
    assert int(st.item()) == 0
    streams = T * k <= 128 or T * k < 10 * E
    rows, flat, worst = g.rows.long(), ids.reshape(-1).long(), 0.0
    for e in torch.unique(flat).tolist()[:32]:
        p = torch.nonzero(flat[rows] == e).reshape(-1)
        worst = max(worst, rel_l2(y[p].cpu(), ffn_plain(x[rows[p] // k], codes[e], scales[e], H, I, group).cpu()))
    assert worst <= (RL2_Y_SMALL if streams else RL2_Y_LARGE), worst


def operators():
    """name -> (call of no arguments, its input to change)"""
    import expert_slot_cache_gb300 as M
    ops = {}
    for name, T, K, N in (("linear_1", 1, 512, 300), ("linear_24", 24, 512, 300), ("linear_parts", 40, 4096, 1024), ("linear_300", 300, 2048, 4096)):
        op = M.W4Linear(M.w4_pack(*(t.to(DEV) for t in draw_w4(K, N, 64, T)), 64), K, N, 64, max_tokens=T)
        x = torch.randn(T, K, device=DEV).to(torch.bfloat16)
        ops[name] = (lambda op=op, x=x, **kw: op.forward(x, **kw), x)
    H, I, E, k = 256, 96, 60, 9
    pool = M.w4_pack_slabs(*draw_experts(H, I, E, 64, 1), H, I, 64)
    for T in (2, 60, 200):
        op = M.W4Experts(pool, H, I, k, E, 64, max_tokens=T)
        x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
        ids, w = draw_routing(T, E, k, T)
        ops[f"experts_{T}"] = (lambda op=op, x=x, ids=ids, w=w, **kw: op.forward(x, ids, w, **kw), x)
        g = M.permute(ids, E)
        ops[f"lists_{T}"] = (lambda g=g, x=x, **kw: M.expert_ffn_w4(x, k, I, E, 64, g.offset, g.rows, g.act_e, g.n_act, E, pool, **kw), x)
    logits = torch.randn(3000, 64, device=DEV)
    ids = torch.topk(logits, 4, dim=1).indices.to(torch.int32)
    ops["balance"] = (lambda **kw: M.balance_loss(logits, ids, 0.1, with_grad=True, **kw).grad, logits)
    return ops


NAMES = ["linear_1", "linear_24", "linear_parts", "linear_300", "experts_2", "experts_60", "experts_200", "lists_2", "lists_60",
         "lists_200", "balance"]


@pytest.mark.parametrize("name", NAMES)
def test_in_a_graph_and_on_a_stream(name):
    call, x = operators()[name]
    first = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for step in range(3):
        x.copy_(torch.randn(x.shape, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call()), step
    assert not torch.equal(first, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = call(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(other, out)


def layer(M, cfg, T, S, sched, layer_no=0):
    H, I, E, group = cfg.H, cfg.I, cfg.E, 64
    codes, scales = draw_experts(H, I, E, group, 10 + layer_no)
    packed = M.w4_pack_slabs(codes, scales, H, I, group)
    host = torch.empty(packed.shape, dtype=torch.uint8, pin_memory=True)
    host.copy_(packed)
    resident = np.random.default_rng(layer_no).permutation(E)[:S].astype(np.int32)
    pool = packed[torch.from_numpy(resident.astype(np.int64)).to(DEV)].contiguous()
    wr = torch.randn(H, E, generator=torch.Generator(device=DEV).manual_seed(layer_no), device=DEV).mul(H ** -0.5).to(torch.bfloat16)
    op = M.SlotCachedMoELayer(wr, pool, cfg.k, I, M.MODE_GATHER, M.POLICY_LRU, host_slabs=host,
                              state=M.CacheState.from_slots(resident, E), max_tokens=T, quant=2, quant_group=group, schedule=sched)
    return op, codes, scales


def test_a_stack_of_4bit_layers_in_one_graph():
    import expert_slot_cache_gb300 as M
    cfg, T = C.TINY, 4
    made = [layer(M, cfg, T, 8, 0, i) for i in range(3)]
    stack = M.LayerStack([m[0] for m in made], T)
    stack._run()
    torch.cuda.synchronize()
    stack.capture()
    g = torch.Generator(device=DEV).manual_seed(3)
    for step in range(4):
        stack.x_all.copy_(torch.randn(stack.x_all.shape, generator=g, device=DEV))
        stack.replay()
        torch.cuda.synchronize()
        for i, (op, codes, scales) in enumerate(made):
            want = experts_plain(stack.xs[i], stack.ids[i], stack.ws[i], codes, scales, cfg.H, cfg.I, 64)
            assert rel_l2(stack.outs[i].double().cpu(), want.cpu()) <= RL2_OUT_BF16, (step, i)
            for s, e in enumerate(op.state.s2e.cpu().tolist()):
                assert torch.equal(op.pool[s].cpu(), op.host_slabs[e])
    assert all(int(m[0].dev_status.item()) == 0 for m in made)


@pytest.mark.parametrize("T,S,sched", [(1, 16, C.SCHED_CHUNKS), (24, 20, C.SCHED_CHUNKS), (24, 20, C.SCHED_WAVES), (90, 20, C.SCHED_WAVES)])
def test_a_larger_layer_from_the_cache(T, S, sched):
    import expert_slot_cache_gb300 as M
    cfg = C.TINY.with_(H=2048, I=768, E=32, k=8, T=T, S=S)
    op, codes, scales = layer(M, cfg, T, S, sched)
    for step in range(2):
        x = torch.randn(T, cfg.H, generator=torch.Generator(device=DEV).manual_seed(step), device=DEV).to(torch.bfloat16)
        r = op.forward(x)
        want = experts_plain(x, r["ids"], r["w"], codes, scales, cfg.H, cfg.I, 64)
        assert rel_l2(r["out"].double().cpu(), want.cpu()) <= RL2_OUT_BF16, step
    assert int(op.dev_status.item()) == 0
