"""Argument checks of group-limited routing and its gradient (no GPU: every refusal returns before any CUDA call)."""
import ctypes

import pytest
import torch

ARG, ALIGN = -1, -3
Z = torch.zeros


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


def test_route(b, p):
    def call(l=p, bf=0, bias=None, mask=None, T=4, E=32, k=2, G=4, g=2, fl=0, ids=p, w=p):
        return b._route_groups(l, bf, bias, mask, T, E, k, G, g, fl, 1.0, ids, w, None)

    assert call(l=None) == ARG and call(ids=None) == ARG and call(w=None) == ARG and call(bf=2) == ARG
    assert call(T=0) == ARG and call(T=(1 << 26) + 1) == ARG and call(E=0) == ARG and call(E=1028) == ARG
    assert call(G=0) == ARG and call(G=5) == ARG and call(G=64, E=64) == ARG and call(g=0) == ARG and call(g=5) == ARG
    assert call(k=0) == ARG and call(k=17) == ARG and call(k=9, g=1) == ARG
    assert call(fl=2) == ARG and call(fl=16) == ARG
    assert call(l=p + 2) == ALIGN and call(l=p + 1, bf=1) == ALIGN


def test_gradient(b, p):
    def call(l=p, bf=0, ids=p, gw=p, T=4, E=32, k=2, fl=0, out=p):
        return b._route_groups_grad(l, bf, ids, gw, T, E, k, fl, 1.0, out, None, None)

    for name in ("l", "ids", "gw", "out"):
        assert call(**{name: None}) == ARG, name
    assert call(T=0) == ARG and call(E=1025) == ARG and call(k=0) == ARG and call(k=17) == ARG and call(bf=3) == ARG
    assert call(fl=2) == ARG and call(fl=4) == ARG
    assert call(l=p + 2) == ALIGN and call(out=p + 2) == ALIGN and call(out=p + 1, bf=1) == ALIGN


def test_python(b):
    i32 = torch.int32
    for bad in (Z(4, 8, dtype=torch.float16), Z(8, 4).t(), Z(4)):
        with pytest.raises(ValueError, match="logits"):
            b.route_groups(bad, 2)
    with pytest.raises(ValueError, match="sel_bias"):
        b.route_groups(Z(4, 8), 2, sel_bias=Z(7))
    with pytest.raises(ValueError, match="token_mask"):
        b.route_groups(Z(4, 8), 2, token_mask=Z(4))
    with pytest.raises(ValueError, match="CUDA device"):
        b.route_groups(Z(4, 8), 2)
    with pytest.raises(ValueError, match="ids"):
        b.route_groups_grad(Z(4, 8), Z(4, 2), Z(4, 2))
    with pytest.raises(ValueError, match="grad_w"):
        b.route_groups_grad(Z(4, 8), Z(4, 2, dtype=i32), Z(4, 3))
    with pytest.raises(ValueError, match="CUDA device"):
        b.route_groups_grad(Z(4, 8), Z(4, 2, dtype=i32), Z(4, 2))
