"""Outputs that lie over inputs in part are refused (no GPU: before any CUDA call)."""
import ctypes

import pytest

ARG = -1


@pytest.fixture(scope="module")
def b():
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as binding
    return binding


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_uint8 * 65536)()
    p.keep = buf
    return (ctypes.addressof(buf) + 255) // 256 * 256


W = 40000  # weights and small arrays, far from the rows


def refused(b, p, x=0, ldx=64, base=None, ldb=32, T=4, K=64, N=32, out=0, ldo=32, f32=0):
    """Whether the forward call refuses these rows (as bytes from p).  L = 0 would be refused behind them, so that nothing
    is ever launched: the call is made with an unaligned A, which comes later."""
    rc = b._adapters(p + x, ldx, None if base is None else p + base, ldb, T, K, N, 8, 2, p + W + 8, p + W, p + W, p + W, p + W, 3, p + out, ldo,
                     f32, None, None, None)
    assert rc in (ARG, -3)
    return rc == ARG


def test_forward(b, p):
    # out (4 rows of 64 bytes) at 8192
    at = dict(x=0, out=8192)
    assert not refused(b, p, **at) and not refused(b, p, base=8192, **at)
    assert not refused(b, p, base=8192 + 256, **at) and not refused(b, p, base=8192 - 256, **at)  # side by side
    for d in (16, 64, 192, 240, -16, -64, -192, -240):
        assert refused(b, p, base=8192 + d, **at), d
    # views of one wider buffer: columns side by side, or not
    wide = dict(x=0, out=8192, ldo=96, ldb=96)
    assert not refused(b, p, base=8192 + 64, **wide) and not refused(b, p, base=8192 + 128, **wide)
    assert not refused(b, p, base=8192 - 64, **wide) and not refused(b, p, base=8192 + 64 + 192, **wide)
    for d in (16, 48, -16, -48, 192, 192 + 48, 192 - 16, 160, -192):
        assert refused(b, p, base=8192 + d, **wide), d
    # other strides over the same range; one row alone has none
    assert refused(b, p, base=8192 + 64, x=0, out=8192, ldo=96, ldb=64) and refused(b, p, base=8192, x=0, out=8192, ldo=96, ldb=32)
    assert not refused(b, p, base=8192 + 64, x=0, out=8192, ldo=96, ldb=64, T=1) and refused(b, p, base=8192 + 32, x=0, out=8192, T=1)
    # x
    for d in (0, 16, 64, 496, -240, -16):
        assert refused(b, p, x=8192, out=8192 + d), d
    assert not refused(b, p, x=8192, out=8192 + 512) and not refused(b, p, x=8192, out=8192 - 256)
    assert not refused(b, p, x=8192, ldx=96, out=8192 + 128, ldo=96) and refused(b, p, x=8192, ldx=96, out=8192 + 112, ldo=96)
    assert not refused(b, p, x=8192, ldx=128, out=8192 + 128, ldo=64, f32=1)  # fp32 rows beside bf16 rows


def test_gradient(b, p):
    def refused(dy=0, ldy=32, x=4096, ldx=64, base=None, ldb=64, dx=8192, lddx=64, weights=True):
        w = p + 20480 if weights else None
        rc = b._adapters_grad(p + dy, ldy, p + x, ldx, p + W, None if base is None else p + base, ldb, 4, 64, 32, 8, 2, p + W + 8, p + W,
                              p + W, p + W, p + W, 3, p + dx, lddx, w, w, p + 32768, 1 << 20, None, None)
        assert rc in (ARG, -3)
        return rc == ARG

    assert not refused() and not refused(base=8192) and not refused(base=8192 + 512)
    for d in (128, 16, -16, -496):
        assert refused(base=8192 + d) and refused(x=8192 + d) and refused(dy=8192 + min(max(d, -240), 496))
    assert refused(dy=8192) and refused(x=8192)
    assert refused(x=8192 + 16, weights=False) is False  # x is not read without da and db
