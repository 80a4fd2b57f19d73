"""The autograd forms record what goes wrong where the caller can read it."""
import pytest
import torch

from tests.test_gpu_adapters import BF, DEV, I32, case, normal

pytestmark = pytest.mark.gpu


def test_adapters():
    import expert_slot_cache_gb300 as M
    for T, lengths in ((3, None), (300, [100, 100, 100]), (64, [8] * 8)):
        x, a, b, scale, ids, starts = case(T, 64, 72, 8, 2, 5, lengths, none=0.0)
        g = torch.Generator(device=DEV).manual_seed(6)
        gy = normal(T, 72, g=g)
        st = torch.zeros(1, dtype=I32, device=DEV)
        leaves = [t.clone().requires_grad_() for t in (x, a, b)]

        def passes():
            st.zero_()
            out = M.AdapterAdd.apply(leaves[0], leaves[1], leaves[2], scale, ids, None, starts, st)
            first = int(st.item())
            st.zero_()
            grads = torch.autograd.grad(out, leaves, gy)
            return first, int(st.item()), [out.detach(), *grads]

        assert passes()[:2] == (0, 0)
        ids[1] = 2
        *codes, bad = passes()
        assert codes == [1, 1]
        ids[1] = -1  # counts as none
        assert all(torch.equal(p, q) for p, q in zip(bad, passes()[2]))
        # without a status: the same results, nothing recorded
        ids[1] = 2
        out = M.AdapterAdd.apply(leaves[0], leaves[1], leaves[2], scale, ids, None, starts)
        assert torch.equal(out.detach(), bad[0])
        if starts is not None:
            ids[1] = 1
            starts[1], starts[2] = starts[2].clone(), starts[1].clone()
            assert passes()[:2] == (4, 4)


def test_a_handle_with_the_callers_status():
    import expert_slot_cache_gb300 as M
    x, a, b, scale, ids, starts = case(300, 64, 72, 8, 2, 5, [100, 100, 100], none=0.0)
    st = torch.zeros(1, dtype=I32, device=DEV)
    one, other = M.Adapters(a, b, scale, st), M.Adapters(b, a, scale, st)
    assert one.dev_status is st and other.dev_status is st
    ids[0] = 7
    one.forward(x, ids, None, starts)
    assert int(st.item()) == 1


def test_routing():
    import expert_slot_cache_gb300 as M
    logits = torch.randn(20, 16, device=DEV, requires_grad=True)
    st = torch.zeros(1, dtype=I32, device=DEV)
    ids, w = M.RouteGroups.apply(logits, 4, 1, 1, None, None, False, False, True, 1.0, st)
    (g,) = torch.autograd.grad(w.sum() * 2, logits, retain_graph=True)
    assert int(st.item()) == 0
    with torch.no_grad():
        ids.data[3, 1] = 16  # the picks that the gradient reads
    torch.autograd.grad(w.sum(), logits)
    assert int(st.item()) == 1
