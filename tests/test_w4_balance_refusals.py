"""Sizes of the packed 4-bit forms and the argument checks of the 4-bit and balance entry points (no GPU: every
refusal returns before any CUDA call)."""
import ctypes

import pytest

ARG, ALIGN = -1, -3


@pytest.fixture(scope="module")
def b():
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as binding
    return binding


@pytest.fixture(scope="module")
def ptr():
    buf = (ctypes.c_uint8 * 8192)()
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    ptr.keep = buf
    return base


def test_sizes(b):
    # 16-column tiles x 64-input blocks of 512 B; a word of two scales per group and column pair; multipliers; 16 B
    assert b.w4_bytes(2048, 768, 128) == 48 * 32 * 512 + 48 * 16 * 32 + 48 * 64 + 16
    assert b.w4_bytes(72, 17, 32) == 2 * 2 * 512 + 2 * 4 * 32 + 2 * 64 + 16
    assert b.w4_bytes(8, 1, 128) == 512 + 32 + 64 + 16
    assert b.w4_slab_bytes(256, 128, 64) == 2 * b.w4_bytes(256, 128, 64) + b.w4_bytes(128, 256, 64)
    for K, N, G in ((0, 8, 64), (12, 8, 64), (64, 0, 64), (64, 8, 16), (64, 8, 0), (1 << 21, 8, 64), (64, 1 << 25, 64)):
        assert b.w4_bytes(K, N, G) == 0
    assert b.w4_slab_bytes(100, 128, 64) == 0 and b.w4_slab_bytes(256, 100, 64) == 0
    assert int(b._balance_ws(8, 16, 0)) == 0 and int(b._balance_ws(8, 1025, 1)) == 0 and int(b._balance_ws(8, 16, 5)) > 0
    assert int(b._experts_w4_ws(0, 256, 128, 2, 16)) == 0 and int(b._experts_w4_ws(4, 256, 128, 17, 32)) == 0


def test_pack_refusals(b, ptr):
    p = ptr
    assert b._w4_pack(None, p, 1, 64, 16, 64, p, None) == ARG
    assert b._w4_pack(p, None, 1, 64, 16, 64, p, None) == ARG
    assert b._w4_pack(p, p, 0, 64, 16, 64, p, None) == ARG
    assert b._w4_pack(p, p, 1, 60, 16, 64, p, None) == ARG
    assert b._w4_pack(p, p, 1, 64, 16, 48, p, None) == ARG
    assert b._w4_pack(p, p, 1, 64, 16, 64, p + 8, None) == ALIGN
    assert b._w4_quantize(None, 1, 64, 16, 64, p, None) == ARG
    assert b._w4_quantize(p, 1, 64, 16, 64, None, None) == ARG
    assert b._w4_pack_slabs(p, p, 1, 100, 128, 64, p, None) == ARG
    assert b._w4_quantize_slabs(p, 1, 256, 100, 64, p, None) == ARG


def test_linear_refusals(b, ptr):
    p = ptr

    def call(x=p, ldx=64, T=1, K=64, N=16, G=64, w=p, out=p, ldo=16, f32=0, ws=p, nws=1 << 20):
        return b._w4_linear(x, ldx, T, K, N, G, w, out, ldo, f32, ws, nws, None, None)

    assert call(x=None) == ARG and call(w=None) == ARG and call(out=None) == ARG
    assert call(T=0) == ARG and call(K=60) == ARG and call(N=0) == ARG and call(G=100) == ARG
    assert call(ldx=56) == ARG and call(ldo=15) == ARG and call(f32=2) == ARG
    assert call(x=p + 2) == ALIGN and call(ldx=68) == ALIGN and call(w=p + 4) == ALIGN
    assert call(out=p + 1) == ALIGN and call(out=p + 2, f32=1) == ALIGN


def test_experts_refusals(b, ptr):
    p = ptr

    def call(x=p, ids=p, w=p, T=4, H=256, I=128, k=2, E=16, G=64, pool=p, S=16, e2s=None, out=p, ws=p, nws=1 << 30):
        return b._experts_w4(x, ids, w, T, H, I, k, E, G, pool, S, e2s, out, ws, nws, None, None)

    for name in ("x", "ids", "w", "pool", "out", "ws"):
        assert call(**{name: None}) == ARG, name
    assert call(T=0) == ARG and call(H=100) == ARG and call(I=100) == ARG and call(k=17) == ARG and call(E=1) == ARG
    assert call(G=16) == ARG and call(S=0) == ARG and call(S=8) == ARG
    assert call(x=p + 2) == ALIGN and call(pool=p + 8) == ALIGN and call(ws=p + 16) == ALIGN and call(nws=64) == ALIGN
    assert call(T=1 << 24) == ARG

    def ffn(y=p, G=64, ws=p, nws=1 << 30, S=16, n=4):
        return b._ffn_w4(p, 4, 256, 128, 2, 16, G, p, p, p, p, n, p, S, None, y, ws, nws, None, None)

    assert ffn(y=None) == ARG and ffn(G=7) == ARG and ffn(S=3) == ARG and ffn(n=-1) == ARG
    assert ffn(y=p + 4) == ALIGN and ffn(ws=p + 16) == ALIGN and ffn(nws=16) == ALIGN


def test_layer_refuses_a_4bit_pool_without_a_group(b, ptr):
    a = b.LayerArgs()
    a.T, a.H, a.E, a.k, a.I, a.S = 4, 256, 16, 2, 128, 16
    for f in ("x", "w_router", "pool", "ids", "w", "out", "workspace"):
        setattr(a, f, ptr)
    a.quant = 2
    assert b._layer(ctypes.byref(a), None, None) == ARG
    a.quant_group = 48
    assert b._layer(ctypes.byref(a), None, None) == ARG


def test_balance_refusals(b, ptr):
    p = ptr

    def call(l=p, bf=0, ids=p, mask=None, seq=None, n_seq=1, T=4, E=16, k=2, fl=0, counts=p, loss=p, grad=None, ws=p,
             nws=1 << 20):
        return b._balance(l, bf, ids, mask, seq, n_seq, T, E, k, fl, 0.1, None, counts, loss, grad, ws, nws, None, None)

    assert call(l=None) == ARG and call(ids=None) == ARG and call(counts=None) == ARG and call(ws=None) == ARG
    assert call(loss=None) == ARG and call(T=0) == ARG and call(E=0) == ARG and call(E=1025) == ARG
    assert call(k=0) == ARG and call(k=17, E=32) == ARG and call(k=3, E=2) == ARG
    assert call(n_seq=0) == ARG and call(n_seq=2) == ARG and call(bf=2) == ARG and call(fl=2) == ARG
    assert call(l=p + 2) == ALIGN and call(ws=p + 8) == ALIGN and call(nws=8) == ALIGN and call(grad=p + 1) == ALIGN


def test_python_refusals(b):
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        b.w4_pack(z(64, 16, dtype=torch.int32), z(1, 16, dtype=torch.bfloat16), 64)
    with pytest.raises(ValueError):
        b.w4_pack(z(64, 16, dtype=torch.uint8), z(2, 16, dtype=torch.bfloat16), 64)
    with pytest.raises(b.MoeError):
        b.W4Linear(z(16, dtype=torch.uint8), 60, 16, 64)
    with pytest.raises(ValueError):
        b.W4Linear(z(16, dtype=torch.uint8), 64, 16, 64)
    op = b.W4Linear(z(b.w4_bytes(64, 16, 64), dtype=torch.uint8), 64, 16, 64, max_tokens=2)
    for x in (z(3, 64, dtype=torch.bfloat16), z(2, 72, dtype=torch.bfloat16), z(2, 64), z(64, 2, dtype=torch.bfloat16).t()):
        with pytest.raises(ValueError):
            op.forward(x)
    with pytest.raises(b.MoeError):
        b.W4Experts(z(16, 8, dtype=torch.uint8), 100, 128, 2, 16, 64)
    ex = b.W4Experts(z(16, b.w4_slab_bytes(256, 128, 64), dtype=torch.uint8), 256, 128, 2, 16, 64, max_tokens=2)
    x, ids, w = z(2, 256, dtype=torch.bfloat16), z(2, 2, dtype=torch.int32), z(2, 2)
    for bad in ((z(3, 256, dtype=torch.bfloat16), ids, w), (x.float(), ids, w), (x, ids.long(), w), (x, ids, w[:1])):
        with pytest.raises(ValueError):
            ex.forward(*bad)
    for bad in ((z(4, 8, dtype=torch.float16), z(4, 2, dtype=torch.int32)), (z(4, 8), z(4, 2)), (z(4, 8), z(3, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            b.balance_loss(*bad, 0.1)
