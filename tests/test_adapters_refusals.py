"""Argument checks of the adapters and their gradients (no GPU: every refusal returns before any CUDA call)."""
import ctypes

import pytest
import torch

ARG, ALIGN = -1, -3
Z, BF, I32 = torch.zeros, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def b():
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as binding
    return binding


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_uint8 * 8192)()
    p.keep = buf
    return (ctypes.addressof(buf) + 255) // 256 * 256


def test_forward(b, p):
    def call(x=p, ldx=64, base=p, ldb=32, T=4, K=64, N=32, R=8, L=2, a=p, w=p, scale=p, ids=p, seq=p, n=3, out=p, ldo=32, f32=0):
        return b._adapters(x, ldx, base, ldb, T, K, N, R, L, a, w, scale, ids, seq, n, out, ldo, f32, None, None, None)

    for name in ("x", "a", "w", "scale", "ids", "out"):
        assert call(**{name: None}) == ARG, name
    assert call(T=0) == ARG and call(T=(1 << 24) + 1) == ARG and call(K=0) == ARG and call(N=0) == ARG
    assert call(R=0) == ARG and call(R=129) == ARG and call(L=0) == ARG and call(L=65536) == ARG
    assert call(n=0) == ARG and call(seq=None, n=3) == ARG and call(f32=2) == ARG
    assert call(ldx=56) == ARG and call(ldo=24) == ARG and call(ldb=24) == ARG
    assert call() == ARG  # out is x
    q = p + 4096
    assert call(out=q, base=q, ldb=40) == ARG and call(n=(1 << 24) + 1) == ARG
    for kw in (dict(K=60), dict(N=30), dict(ldx=68), dict(ldo=36), dict(ldb=36), dict(x=p + 2), dict(out=q + 8), dict(base=p + 8),
               dict(a=p + 8), dict(w=p + 8), dict(ldo=34, f32=1)):
        assert call(**dict(dict(out=q), **kw)) == ALIGN, kw


def test_gradient(b, p):
    def call(dy=p, ldy=32, x=p, ldx=64, kept=p, base=p, ldb=64, T=4, K=64, N=32, R=8, L=2, a=p, w=p, scale=p, ids=p, seq=p, n=3,
             dx=p, lddx=64, da=p, db=p, ws=p, nws=1 << 20):
        return b._adapters_grad(dy, ldy, x, ldx, kept, base, ldb, T, K, N, R, L, a, w, scale, ids, seq, n, dx, lddx, da, db, ws, nws,
                                None, None)

    for name in ("dy", "x", "kept", "a", "w", "scale", "ids", "ws", "da", "db"):
        assert call(**{name: None}) == ARG, name
    assert call(dx=None, da=None, db=None) == ARG
    assert call(T=0) == ARG and call(R=129) == ARG and call(L=0) == ARG and call(seq=None) == ARG
    assert call(ldy=24) == ARG and call(ldx=56) == ARG and call(ldb=56) == ARG and call(lddx=56) == ARG
    q = p + 4096
    assert call(dy=q) == ARG and call(x=q) == ARG  # dx is x, dx is dy
    assert call(dx=q, base=q, ldb=72) == ARG
    for kw in (dict(K=60), dict(dy=p + 2), dict(dx=q + 8), dict(da=p + 4), dict(ws=p + 16), dict(nws=16)):
        assert call(**dict(dict(dx=q), **kw)) == ALIGN, kw
    assert int(b._adapters_grad_ws(0, 8)) == 0 and int(b._adapters_grad_ws(4, 129)) == 0 and int(b._adapters_grad_ws(4, 8)) >= 128


def test_python(b):
    a, w, s = Z(2, 8, 64, dtype=BF), Z(2, 8, 32, dtype=BF), Z(2)
    for bad in ((a[0], w, s), (a, w[:, :4], s), (a.float(), w, s), (a, w, Z(3)), (a, w, s.double()), (a[:, :, :60].contiguous(), w, s),
                (Z(1, 129, 64, dtype=BF), Z(1, 129, 32, dtype=BF), Z(1)), (a.transpose(0, 1), w.transpose(0, 1), Z(8))):
        with pytest.raises(ValueError):
            b.Adapters(*bad)
    op = b.Adapters(a, w, s)
    x, ids, starts = Z(4, 64, dtype=BF), Z(2, dtype=I32), Z(3, dtype=I32)
    calls = [dict(x=x.float()), dict(x=Z(4, 72, dtype=BF)), dict(ids=ids.long()), dict(ids=Z(3, dtype=I32)), dict(seq_start=None),
             dict(seq_start=Z(3)), dict(base=Z(4, 33, dtype=BF)), dict(base=Z(4, 32, dtype=torch.float16)), dict(kept=Z(4, 9)),
             dict(out=Z(4, 32)), dict()]
    for kw in calls:
        args = dict(dict(x=x, ids=ids, seq_start=starts, base=Z(4, 32, dtype=BF)), **kw)
        with pytest.raises(ValueError):
            op.forward(**args)
    dy, kept = Z(4, 32, dtype=BF), Z(4, 8)
    for kw in (dict(dy=dy.float()), dict(x=None), dict(kept=None), dict(kept=Z(4, 7)), dict(base=dy), dict(ids=ids.long()), dict()):
        args = dict(dict(dy=dy, x=x, kept=kept, ids=ids, seq_start=starts), **kw)
        with pytest.raises(ValueError):
            op.grad(**args)
    lin = b.W4Linear(Z(b.w4_bytes(64, 48, 64), dtype=torch.uint8), 64, 48, 64, max_tokens=4)
    with pytest.raises(ValueError, match="adapters"):
        lin.forward(x, adapters=op, adapter_ids=ids, seq_start=starts)
    with pytest.raises(ValueError, match="base"):
        b.AdapterAdd.apply(x, a, w, s, ids, Z(4, 32), starts)
