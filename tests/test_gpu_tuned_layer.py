"""A tuned 4-bit layer as it is served and trained: a 4-bit projection with adapters of many requests, a router with
groups and a balance bias, 4-bit experts, the balance loss."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV, BF, I32, F64 = "cuda", torch.bfloat16, torch.int32, torch.float64
H, I, E, K, R, L, GROUP = 256, 128, 32, 4, 12, 5, 64


def layer(seed=1, tokens=64):
    import expert_slot_cache_gb300 as M
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, size=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * size

    proj = normal(H, H, size=H ** -0.5).to(BF)
    lin = M.W4Linear(M.w4_quantize(proj, GROUP), H, H, GROUP, max_tokens=tokens)
    ex = M.W4Experts(M.w4_quantize_slabs(normal(E, 3 * H * I, size=H ** -0.5).to(BF), H, I, GROUP), H, I, K, E, GROUP, max_tokens=tokens)
    a, b = normal(L, R, H, size=H ** -0.5).to(BF), normal(L, R, H, size=0.1).to(BF)
    scale = torch.rand(L, generator=g, device=DEV) + 0.5
    wr = normal(H, E, size=H ** -0.5)
    bias = torch.round(normal(E) * 30) * 0.001
    return lin, ex, a, b, scale, wr, bias, normal


def test_decoding_in_a_graph():
    """One step for 24 requests, captured and replayed with other inputs, requests and adapters' weights."""
    import expert_slot_cache_gb300 as M
    lin, ex, a, b, scale, wr, bias, normal = layer()
    op = M.Adapters(a, b, scale)
    x, ids = normal(24, H).to(BF), torch.arange(24, dtype=I32, device=DEV) % (L + 1) - 1

    def step():
        h = lin.forward(x, adapters=op, adapter_ids=ids)
        r = M.route_groups(h.float() @ wr, K, 8, 3, sel_bias=bias, sigmoid=True, scale=2.5)
        return h, r.ids, r.w, ex.forward(h, r.ids, r.w)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # cuBLAS sets itself up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        x.copy_(normal(24, H))
        ids.copy_(torch.roll(ids, 1))
        a.copy_(normal(L, R, H, size=H ** -0.5))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        h, eid, w, y = got
        plain = lin.forward(x).double()
        for t in range(24):
            l = int(ids[t])
            if l >= 0:
                plain[t] += scale[l].double() * (x[t].double() @ a[l].double().T) @ b[l].double()
        # the projection's result is rounded before the adapters' part is added: two roundings (and fp32 sums)
        assert bool(((h.double() - plain).abs() <= 2 * 2.0 ** -8 * plain.abs() + 1e-3).all())
        assert bool((w.sum(1) - 2.5).abs().max() < 1e-4) and bool(((eid >= 0) & (eid < E)).all())
        for row in eid.cpu().numpy():
            assert len(set(row)) == K and len(set(row // (E // 8))) <= 3
        assert bool(y.isfinite().all())
    assert int(op.dev_status.item()) == 0 and int(lin.dev_status.item()) == 0 and int(ex.dev_status.item()) == 0


def test_training_step():
    """Adapters, router weights and the balance loss in one graph; gradients against fp64 autograd of the formulas.

    The gradient reaches the adapters in bf16 (half a step of 2^-8 of each value), a, b and their gradients are rounded
    once more: relative errors of some 2^-8 whose signs are random, so below 1e-2 of the gradient's norm."""
    import expert_slot_cache_gb300 as M
    lin, _, a, b, scale, wr, bias, normal = layer(3, tokens=700)
    T = 700
    starts = torch.tensor([0, 250, 250, 256, 700], dtype=I32, device=DEV)
    ids = torch.tensor([2, 1, -1, 0], dtype=I32, device=DEV)
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    mask[690:] = False
    x = normal(T, H).to(BF)
    base = lin.forward(x)
    gw = normal(T, K)
    leaves = [t.clone().requires_grad_() for t in (x, a, b, wr, base)]

    def loss_of(h, logits, eid, w):
        lb, _ = M.BalanceLoss.apply(logits, eid, 0.5, starts, mask)
        return (w * gw).sum() / T + lb + (h.float() ** 2).sum() * 1e-3 / T

    h = M.AdapterAdd.apply(leaves[0], leaves[1], leaves[2], scale, ids, leaves[4], starts)
    logits = h.float() @ leaves[3]
    eid, w = M.RouteGroups.apply(logits, K, 8, 3, bias, mask, True, False, True, 2.5)
    loss = loss_of(h, logits, eid, w)
    grads = torch.autograd.grad(loss, leaves)

    p = [t.double().clone().requires_grad_() for t in (x, a, b, wr, base)]
    parts = []
    for (s, e), l in zip(((0, 250), (250, 250), (250, 256), (256, 700)), ids.tolist()):
        parts.append(p[4][s:e] + (scale[l].double() * (p[0][s:e] @ p[1][l].T) @ p[2][l] if l >= 0 else 0))
    h64 = torch.cat(parts)
    h64 = h64 + (h.detach().double() - h64.detach())  # the values as they were rounded
    l64 = h64 @ p[3]
    s = torch.sigmoid(l64.gather(1, eid.clamp(min=0).long()))
    w64 = torch.where(mask[:, None], 2.5 * s / s.sum(1, keepdim=True), 0.0)
    prob = torch.softmax(l64, 1)
    lb = 0.0
    for s0, e0 in ((0, 250), (250, 250), (250, 256), (256, 700)):
        t = torch.arange(s0, e0, device=DEV)[mask[s0:e0]]
        if len(t):
            f = torch.bincount(eid[t].reshape(-1).long(), minlength=E).double() * E / (K * len(t))
            lb = lb + 0.5 / int(mask.sum()) * (prob[t] * f).sum()
    want = (w64 * gw.double()).sum() / T + lb + (h64 ** 2).sum() * 1e-3 / T
    assert abs(loss.item() - want.item()) <= 1e-4 * abs(want.item()) + 1e-5
    for name, got, ref in zip(("x", "a", "b", "wr", "base"), grads, torch.autograd.grad(want, p)):
        err = (got.double() - ref).norm() / ref.norm()
        assert float(err) <= 1e-2, (name, float(err))


def test_backward_in_a_graph():
    """The gradients of a captured step, replayed, equal those of an eager one."""
    import expert_slot_cache_gb300 as M
    _, _, a, b, scale, wr, bias, normal = layer(5)
    x, base, gy = normal(300, H).to(BF), normal(300, H).to(BF), normal(300, K)
    starts = torch.tensor([0, 120, 300], dtype=I32, device=DEV)
    ids = torch.tensor([1, 4], dtype=I32, device=DEV)
    op = M.Adapters(a, b, scale)
    kept = torch.empty(300, R, device=DEV)
    logits = normal(300, E)

    def step():
        h = op.forward(x, ids, base, starts, kept=kept)
        r = M.route_groups(logits, K, 8, 3, sel_bias=bias, sigmoid=True)
        gl = M.route_groups_grad(logits, r.ids, gy, sigmoid=True)
        return [h, gl, *op.grad(h, x, kept, ids, None, starts)]

    step()
    graphs = []
    for _ in range(2):  # two graphs: neither has the other's workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    for seed in range(2):
        x.copy_(normal(300, H))
        logits.copy_(normal(300, E))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in held] for _, held in graphs]
        want = step()
        for one in got:
            assert all(torch.equal(p, q) for p, q in zip(one, want))
