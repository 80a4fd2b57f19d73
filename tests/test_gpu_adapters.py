"""Low-rank adapters and their gradients against the formulas in 64 bits.

Tolerances.  Products of bf16 values are exact in fp32, and a sum of n of them in any order, each addition off by at
most 2^-23 of what it adds up, is within n 2^-23 of the sum of the terms' sizes.  So v (and dv) is within
(K + 2) 2^-23 of s |x| |A|^T.  v takes part in the second product with 16 significant bits or more (2^-16 of a term),
which adds R 2^-23 of |v| |B|; the result is rounded once (half a step: bf16 2^-8, fp32 2^-24).  dA and dB take v and
dv with 24 bits: (rows + 2) 2^-23 of |dv|^T |x|, and what dv itself is off by.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV, BF, I32, F64 = "cuda", torch.bfloat16, torch.int32, torch.float64
U = 2.0 ** -23


def normal(*shape, g, dtype=BF, size=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * size).to(dtype)


def case(T, K, N, R, L, seed, lengths=None, none=0.15, lead=0):
    """x, a, b, scale, ids, seq_start (None: a row each)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    n = T if lengths is None else len(lengths)
    ids = r.integers(0, L, n).astype(np.int32)
    ids[r.random(n) < none] = -1
    starts = None if lengths is None else torch.from_numpy((lead + np.concatenate([[0], np.cumsum(lengths)])).astype(np.int32)).to(DEV)
    return (normal(T, K, g=g), normal(L, R, K, g=g, size=K ** -0.5), normal(L, R, N, g=g, size=0.1),
            torch.rand(L, generator=g, device=DEV) + 0.5, torch.from_numpy(ids).to(DEV), starts)


def rows_of(T, ids, starts):
    """(first, end, adapter) of the sequences with an adapter."""
    ids = ids.cpu().tolist()
    s = list(range(T + 1)) if starts is None else starts.cpu().tolist()
    return [(p, q, l) for p, q, l in zip(s, s[1:], ids) if q > p and l >= 0]


def shrink(x, w, scale, spans):
    """s_l x W_l^T and its error bound."""
    v = torch.zeros(x.shape[0], w.shape[1], dtype=F64, device=DEV)
    e = torch.zeros_like(v)
    for p, q, l in spans:
        v[p:q] = scale[l].double() * (x[p:q].double() @ w[l].double().T)
        e[p:q] = (x.shape[1] + 2) * U * scale[l].double() * (x[p:q].double().abs() @ w[l].double().abs().T)
    return v, e


def expand(v, e, w, base, spans, dtype):
    """base + v W_l and its error bound."""
    T, N = v.shape[0], w.shape[2]
    out = torch.zeros(T, N, dtype=F64, device=DEV) if base is None else base.double()
    tol = torch.zeros(T, N, dtype=F64, device=DEV)
    for p, q, l in spans:
        size = w[l].double().abs()
        out[p:q] += v[p:q] @ w[l].double()
        tol[p:q] = e[p:q] @ size + (2.0 ** -16 + (w.shape[1] + 2) * U) * (v[p:q].abs() @ size)
    if base is not None:
        tol += 2 * U * base.double().abs()
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    return out, tol + half * (out.abs() + tol) + 1e-38


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: {float((err / tol).nan_to_num(9e9).max())}"


def check(T, K, N, R, L, seed, lengths=None, dtype=BF, with_base=True, grads=True, **kw):
    import expert_slot_cache_gb300 as M
    x, a, b, scale, ids, starts = case(T, K, N, R, L, seed, lengths, **kw)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    base = normal(T, N, g=g, dtype=dtype) if with_base else None
    op = M.Adapters(a, b, scale)
    kept = torch.full((T, R), float("nan"), device=DEV)
    out = op.forward(x, ids, base, starts, out_dtype=dtype, kept=kept)
    spans = rows_of(T, ids, starts)
    v, e = shrink(x, a, scale, spans)
    close(kept, v, e, "kept")
    want, tol = expand(v, e, b, base, spans, dtype)
    close(out, want, tol, "out")
    again = op.forward(x, ids, base, starts, out_dtype=dtype)
    assert torch.equal(out, again)
    if with_base:
        same = base.clone()
        assert op.forward(x, ids, same, starts, out=same) is same and torch.equal(same, out)
    outside = torch.ones(T, dtype=torch.bool, device=DEV)
    for p, q, _ in spans:
        outside[p:q] = False
    assert not bool(kept[outside].any())
    if with_base:
        assert torch.equal(out[outside], base[outside])
    if grads:
        dy, dx0 = normal(T, N, g=g, size=0.1), normal(T, K, g=g, size=0.1) if with_base else None
        r = op.grad(dy, x, kept, ids, dx0, starts)
        dv, de = shrink(dy, b, scale, spans)
        want, tol = expand(dv, de, a, dx0, spans, BF)
        close(r.dx, want, tol, "dx")
        for got, lhs, err, rhs, name in ((r.da, dv, de, x, "da"), (r.db, kept.double(), 0 * e, dy, "db")):
            want = torch.zeros(got.shape, dtype=F64, device=DEV)
            size, off, n = torch.zeros_like(want), torch.zeros_like(want), [0] * L
            for p, q, l in spans:
                want[l] += lhs[p:q].T @ rhs[p:q].double()
                size[l] += lhs[p:q].abs().T @ rhs[p:q].double().abs()
                off[l] += err[p:q].T @ rhs[p:q].double().abs()
                n[l] += q - p
            n = torch.tensor(n, device=DEV).view(L, 1, 1)
            close(got, want, off + (n + 2) * U * size + 1e-38, name)
        twice = op.grad(dy, x, kept, ids, dx0, starts)
        assert torch.equal(r.dx, twice.dx) and torch.equal(r.da, twice.da) and torch.equal(r.db, twice.db)
        alone = op.grad(dy, None, None, ids, dx0, starts, with_weights=False)
        assert alone.da is None and torch.equal(alone.dx, r.dx)
        alone = op.grad(dy, x, kept, ids, None, starts, with_dx=False)
        assert alone.dx is None and torch.equal(alone.da, r.da) and torch.equal(alone.db, r.db)
    assert int(op.dev_status.item()) == 0


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T,K,N,R,L", [(1, 8, 8, 1, 1), (1, 2048, 2048, 16, 8), (3, 72, 40, 3, 2), (2, 1416, 1000, 24, 3), (64, 256, 512, 16, 64),
                                       (33, 520, 264, 100, 5), (17, 4096, 136, 128, 2), (5, 64, 4096, 8, 1), (200, 128, 64, 17, 9)])
def test_a_row_each(T, K, N, R, L, dtype):
    check(T, K, N, R, L, T + K, dtype=dtype)


@pytest.mark.parametrize("T,K,N,R", [(2, 64, 64, 16), (9, 72, 200, 8), (31, 136, 520, 33), (128, 128, 128, 16), (129, 264, 136, 64), (300, 2048, 2048, 8),
                                     (1000, 1416, 1000, 24), (520, 512, 1032, 128), (4096, 256, 384, 64), (777, 8, 8, 1), (640, 4096, 64, 97)])
def test_one_sequence(T, K, N, R):
    check(T, K, N, R, 2, T + R, lengths=[T], none=0.0)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("lengths,K,N,R,L", [([1, 1, 1, 1, 100, 37], 1416, 1000, 24, 3), ([0, 5, 0, 0, 300, 1, 64, 128, 129, 2], 256, 264, 16, 2),
                                             ([16] * 40, 136, 128, 8, 5), ([700, 3, 1, 500], 520, 136, 64, 1), ([9] * 7 + [0, 0], 64, 72, 128, 4),
                                             ([1] * 150 + [333] + [0] * 5 + [8] * 20, 128, 256, 31, 12), ([65, 63, 64, 1, 127], 2048, 4096, 16, 2)])
def test_packed_sequences(lengths, K, N, R, L, dtype):
    check(sum(lengths), K, N, R, L, K + len(lengths), lengths=lengths, dtype=dtype)
    check(sum(lengths), K, N, R, L, K + 1, lengths=lengths, dtype=dtype, with_base=False)


def test_rows_outside_the_sequences():
    check(500, 128, 264, 16, 2, 1, lengths=[40, 200, 7], lead=31, none=0.0)
    check(40, 128, 136, 8, 2, 2, lengths=[3], lead=20, none=0.0)
    check(300, 64, 64, 8, 1, 3, lengths=[0, 0], lead=300, none=0.0)
    check(300, 64, 64, 8, 3, 4, lengths=[0], lead=0, none=0.0)
    check(700, 72, 520, 8, 3, 5, lengths=[100, 300], lead=150, none=1.0)


def test_many_sequences_and_adapters():
    r = np.random.default_rng(7)
    check(3000, 64, 72, 4, 300, 8, lengths=r.multinomial(3000, np.ones(700) / 700).tolist())
    check(2500, 64, 72, 8, 2, 9, lengths=[0] * 1200 + [1] * 500 + [2000] + [0] * 900, none=0.3)


@pytest.mark.parametrize("R", [16, 32, 64, 80, 128])
def test_many_passes_over_long_sequences(R):
    """Rings of every number of slots, many rounds, passes one behind the other: the same bits each time, no timeout."""
    import expert_slot_cache_gb300 as M
    lengths = [1900, 70, 3000, 1030]
    x, a, b, scale, ids, starts = case(6000, 512, 264, R, 2, R, lengths, none=0.0)
    g = torch.Generator(device=DEV).manual_seed(4)
    dy, base = normal(6000, 264, g=g), normal(6000, 264, g=g)
    op = M.Adapters(a, b, scale)
    kept = torch.empty(6000, R, device=DEV)
    out = op.forward(x, ids, base, starts, kept=kept)
    want = op.grad(dy, x, kept, ids, None, starts)
    passes = [(op.forward(x, ids, base, starts), op.grad(dy, x, kept, ids, None, starts)) for _ in range(40)]
    assert all(torch.equal(o, out) and all(torch.equal(p, q) for p, q in zip(r, want)) for o, r in passes)
    assert int(op.dev_status.item()) == 0


def test_a_thousand_gradients():
    """A ring of three slots, tiles with rows to be cleared among others, launches that overlap: no wait gives up."""
    import expert_slot_cache_gb300 as M
    lengths = [1261, 0, 996, 567, 1068, 19, 1740, 236, 759, 409, 1137]
    for R, K, N, L in ((32, 2048, 4096, 3), (24, 264, 136, 2), (48, 512, 512, 1)):
        x, a, b, scale, ids, starts = case(8192, K, N, R, L, 7, lengths, none=0.0)
        g = torch.Generator(device=DEV).manual_seed(8)
        dy, kept = normal(8192, N, g=g, size=0.01), torch.empty(8192, R, device=DEV)
        op = M.Adapters(a, b, scale)
        op.forward(x, ids, None, starts, kept=kept)
        want = op.grad(dy, x, kept, ids, None, starts)
        off = torch.zeros((), dtype=torch.int64, device=DEV)
        for i in range(340):
            r = op.grad(dy, x, kept, ids, None, starts)
            off += sum((p != q).sum() for p, q in zip(r, want))
            if i % 50 == 0:
                assert int(op.dev_status.item()) == 0  # (stops here, should a wait have given up)
        assert int(off) == 0 and int(op.dev_status.item()) == 0


def test_large_values_and_other_rows_nan():
    """NaN and infinities stay in their rows, whatever the tile; rows of no sequence are not read into anything."""
    import expert_slot_cache_gb300 as M
    for lengths, lead in (([70, 1, 200, 3], 9), ([1] * 20, 2), ([300], 30)):
        T = sum(lengths) + 2 * lead
        x, a, b, scale, ids, starts = case(T, 264, 520, 24, 2, 3, lengths, none=0.0, lead=lead)
        g = torch.Generator(device=DEV).manual_seed(4)
        dy, base = normal(T, 520, g=g), normal(T, 520, g=g)
        op = M.Adapters(a, b, scale)
        kept = torch.empty(T, 24, device=DEV)
        want = op.forward(x, ids, base, starts, kept=kept)
        grad = op.grad(dy, x, kept, ids, None, starts)
        bad, dbad, kbad = x.clone(), dy.clone(), kept.clone()
        for t in (0, lead - 1, T - 1, T - lead):  # in no sequence
            bad[t], dbad[t], kbad[t] = float("nan"), float("inf"), float("nan")
        got = op.grad(dbad, bad, kbad, ids, None, starts)
        assert torch.equal(got.da, grad.da) and torch.equal(got.db, grad.db) and torch.equal(got.dx, grad.dx)
        hit = lead + 5
        bad[hit, 3] = float("inf")
        out = op.forward(bad, ids, base, starts)
        ok = torch.arange(T, device=DEV) != hit
        assert torch.equal(out[ok], want[ok]) and not bool(out[hit].isfinite().any())
        x2 = x * 1e30  # v about 1e30: the parts of v must not overflow on their way
        out = op.forward(x2, ids, None, starts, out_dtype=torch.float32)
        spans = rows_of(T, ids, starts)
        v, e = shrink(x2, a, scale, spans)
        w, tol = expand(v, e, b, None, spans, torch.float32)
        close(out, w, tol, "large")


def test_infinite_products_keep_their_sign():
    import expert_slot_cache_gb300 as M
    for T in (1, 300):
        x = torch.zeros(T, 64, dtype=BF, device=DEV)
        x[:, 0] = float("inf")
        a, b = torch.zeros(1, 8, 64, dtype=BF, device=DEV), torch.ones(1, 8, 64, dtype=BF, device=DEV)
        a[:, :, 0] = 1.0
        b[:, :, ::2] = -1.0
        op = M.Adapters(a, b, torch.ones(1, device=DEV))
        out = op.forward(x.clone(), torch.zeros(1, dtype=I32, device=DEV), None, torch.tensor([0, T], dtype=I32, device=DEV))
        assert bool((out[:, 1::2] == float("inf")).all()) and bool((out[:, ::2] == float("-inf")).all())


def test_strided_rows():
    import expert_slot_cache_gb300 as M
    for T, lengths in ((6, None), (200, [150, 50])):
        x, a, b, scale, ids, starts = case(T, 128, 72, 8, 3, 5, lengths)
        g = torch.Generator(device=DEV).manual_seed(6)
        base = normal(T, 72, g=g)
        op = M.Adapters(a, b, scale)
        want = op.forward(x, ids, base, starts)
        wide = torch.full((T, 128 + 24), float("nan"), dtype=BF, device=DEV)
        wide[:, 8:136] = x
        bw = torch.full((T, 96), float("nan"), dtype=BF, device=DEV)
        bw[:, 16:88] = base
        ow = torch.full((T, 88), 7.0, dtype=BF, device=DEV)
        out = op.forward(wide[:, 8:136], ids, bw[:, 16:88], starts, out=ow[:, 8:80])
        assert torch.equal(out, want) and bool((ow[:, :8] == 7).all()) and bool((ow[:, 80:] == 7).all())
        dy, kept = normal(T, 72, g=g), torch.empty(T, 8, device=DEV)
        op.forward(x, ids, base, starts, kept=kept)
        dw = torch.full((T, 80), float("nan"), dtype=BF, device=DEV)
        dw[:, :72] = dy
        r, s = op.grad(dy, x, kept, ids, None, starts), op.grad(dw[:, :72], wide[:, 8:136], kept, ids, None, starts)
        assert torch.equal(r.dx, s.dx) and torch.equal(r.da, s.da) and torch.equal(r.db, s.db)


def test_bad_ids_and_starts():
    """An id that is no adapter counts as none and is flagged; starts that descend are flagged and stay in bounds."""
    import expert_slot_cache_gb300 as M
    x, a, b, scale, ids, starts = case(300, 64, 72, 8, 2, 5, [100, 100, 100], none=0.0)
    g = torch.Generator(device=DEV).manual_seed(6)
    base, dy = normal(300, 72, g=g), normal(300, 72, g=g)
    op = M.Adapters(a, b, scale)
    kept = torch.empty(300, 8, device=DEV)
    for bad in (2, -2, 1 << 30):
        ids[1] = bad
        out = op.forward(x, ids, base, starts, kept=kept)
        assert torch.equal(out[100:200], base[100:200]) and int(op.dev_status.item()) == 1
        r = op.grad(dy, x, kept, ids, None, starts)
        assert not bool(r.dx[100:200].any())
        op.dev_status.zero_()
    ids[1] = 1
    for wrong in ([0, 200, 100, 300], [-50, 100, 200, 4000], [250, 200, 100, 0]):
        op.forward(x, ids, base, torch.tensor(wrong, dtype=I32, device=DEV), kept=kept)
        op.grad(dy, x, kept, ids, None, torch.tensor(wrong, dtype=I32, device=DEV))
        torch.cuda.synchronize()
        assert int(op.dev_status.item()) == (4 if wrong[1] > wrong[2] else 0)
        op.dev_status.zero_()


def test_autograd_against_the_formula_and_differences():
    import expert_slot_cache_gb300 as M
    x, a, b, scale, ids, starts = case(60, 64, 72, 8, 3, 9, [20, 1, 39], none=0.0)
    g = torch.Generator(device=DEV).manual_seed(6)
    base, gw = normal(60, 72, g=g), normal(60, 72, g=g)
    leaves = [t.clone().requires_grad_() for t in (x, a, b, base)]
    out = M.AdapterAdd.apply(leaves[0], leaves[1], leaves[2], scale, ids, leaves[3], starts)
    grads = torch.autograd.grad(out, leaves, gw, create_graph=True)
    assert torch.equal(grads[3].detach(), gw)
    op = M.Adapters(a, b, scale)
    kept = torch.empty(60, 8, device=DEV)
    op.forward(x, ids, base, starts, kept=kept)
    r = op.grad(gw, x, kept, ids, None, starts)
    assert torch.equal(grads[0].detach(), r.dx) and torch.equal(grads[1].detach(), r.da.to(BF)) and torch.equal(grads[2].detach(), r.db.to(BF))
    with pytest.raises(RuntimeError, match="second derivative"):
        (grads[1].float() ** 2).sum().backward()
    # a scalar loss over everything: the gradient that arrives is one value with strides of 0
    (only,) = torch.autograd.grad(M.AdapterAdd.apply(x, leaves[1], b, scale, ids, None, starts).sum(), leaves[1])
    ones = op.grad(torch.ones_like(gw), x, kept, ids, None, starts)
    assert torch.equal(only, ones.da.to(BF))
    # differences: the loss is bilinear in a and b, so a central difference in one entry is exact but for its rounding
    spans = rows_of(60, ids, starts)

    def loss(av, bv):
        v, _ = shrink(x, av, scale, spans)
        return float((expand(v, v * 0, bv, base, spans, torch.float32)[0] * gw.double()).sum())

    for l, i, k in ((0, 0, 0), (1, 7, 63), (2, 3, 11)):
        for w, got in ((a, r.da), (b, r.db)):
            h = 0.25
            up, down = w.double().clone(), w.double().clone()
            up[l, i, k] += h
            down[l, i, k] -= h
            args = [(up, b), (down, b)] if w is a else [(a, up), (a, down)]
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            assert abs(float(got[l, i, k]) - diff) <= 1e-3 * abs(diff) + 1e-4


def test_streams_and_graphs():
    import expert_slot_cache_gb300 as M
    for T, lengths in ((8, None), (300, [100, 1, 199])):
        x, a, b, scale, ids, starts = case(T, 256, 264, 16, 3, 9, lengths, none=0.0)
        g = torch.Generator(device=DEV).manual_seed(6)
        base, dy = normal(T, 264, g=g), normal(T, 264, g=g)
        op = M.Adapters(a, b, scale)
        kept = torch.empty(T, 16, device=DEV)

        def step(stream=None):
            out = op.forward(x, ids, base, starts, kept=kept, stream=stream)
            return [out, *op.grad(dy, x, kept, ids, None, starts, stream=stream)]

        want = step()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = step(s)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for seed in (1, 2):
            g2 = torch.Generator(device=DEV).manual_seed(seed)
            x.copy_(normal(T, 256, g=g2))
            a.copy_(normal(3, 16, 256, g=g2, size=0.1))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in held]
            want = step()
            assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_beside_a_4bit_projection():
    """W4Linear with adapters: the projection's result plus the adapters' part, in its buffer."""
    import expert_slot_cache_gb300 as M
    for T, lengths, dtype in ((5, None, BF), (70, [30, 40], torch.float32), (200, [150, 50], BF)):
        x, a, b, scale, ids, starts = case(T, 256, 520, 16, 3, 9, lengths)
        g = torch.Generator(device=DEV).manual_seed(6)
        lin = M.W4Linear(M.w4_quantize(normal(256, 520, g=g, size=0.1), 64), 256, 520, 64, max_tokens=T, out_dtype=dtype)
        op = M.Adapters(a, b, scale)
        plain = lin.forward(x)
        out = torch.empty(T, 520, dtype=dtype, device=DEV)
        got = lin.forward(x, out=out, adapters=op, adapter_ids=ids, seq_start=starts)
        assert got is out and torch.equal(got, op.forward(x, ids, plain, starts))
        assert torch.equal(lin.forward(x, adapters=op, adapter_ids=ids, seq_start=starts), got)
        with pytest.raises(ValueError, match="adapter_ids"):
            lin.forward(x, adapters=op)
        with pytest.raises(ValueError, match="ids"):
            lin.forward(x, adapters=op, adapter_ids=ids[:-1], seq_start=starts)
