"""Gradients that arrive in rows of every kind: contiguous but on any address, strided, one value for all."""
import pytest
import torch

from tests.test_gpu_adapters import BF, DEV, case, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,lengths", [(1, None), (5, None), (200, [150, 50])])
def test_gradients_of_any_layout(T, lengths):
    import expert_slot_cache_gb300 as M
    x, a, b, scale, ids, starts = case(T, 64, 72, 8, 2, 5, lengths, none=0.0)
    leaves = [t.clone().requires_grad_() for t in (x, a, b)]
    gy = normal(T, 72, g=torch.Generator(device=DEV).manual_seed(6))
    out = M.AdapterAdd.apply(leaves[0], leaves[1], leaves[2], scale, ids, None, starts)
    want = torch.autograd.grad(out, leaves, gy, retain_graph=True)
    buf = torch.full((T * 100 + 64,), float("nan"), dtype=BF, device=DEV)
    for view in (buf[1:1 + T * 72].view(T, 72), buf[3:3 + T * 72].view(T, 72), buf[:T * 72].view(T, 72), buf[:T * 80].view(T, 80)[:, 8:],
                 buf[:T * 90].view(T, 90)[:, 5:77], buf[:T * 72].view(72, T).t()):
        view.copy_(gy)
        got = torch.autograd.grad(out, leaves, view, retain_graph=True)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        buf.fill_(float("nan"))
    # a flat buffer of several tensors, as a parameter store makes one
    flat = torch.cat([torch.zeros(3, dtype=BF, device=DEV), out.reshape(-1)])
    weight = torch.cat([torch.ones(3, dtype=BF, device=DEV), gy.reshape(-1)])
    got = torch.autograd.grad((flat * weight).float().sum(), leaves)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
