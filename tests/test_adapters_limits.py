"""The gradients' limit on adapters x sequences x features (no GPU: before any CUDA call)."""
import ctypes

import pytest

ARG, ALIGN = -1, -3


@pytest.mark.parametrize("L,n,K,N,ok", [(65535, 65536, 2048, 2048, True), (65535, 65537, 2048, 2048, True), (65535, 65538, 2048, 2048, False), (64, 1 << 24, 2048, 2048, True),
                                        (256, 1 << 24, 2048, 2048, True), (257, 1 << 24, 2048, 2048, False), (65535, 1 << 24, 8, 8, True),
                                        (65535, 1 << 24, 16, 8, False)])
def test_work(L, n, K, N, ok):
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as b
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 255) // 256 * 256

    def call(weights):  # an unaligned A, so that nothing is launched
        w = p if weights else None
        return b._adapters_grad(p, N, p + (1 << 32), K, p, None, 0, 4, K, N, 8, L, p + 8, p, p, p, p, n, p + (1 << 34), K, w, w, p, 1 << 40, None, None)

    assert call(True) == (ALIGN if ok else ARG) and call(False) == ALIGN
