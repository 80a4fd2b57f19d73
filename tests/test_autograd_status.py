"""The autograd forms hand the caller's status to the library (no GPU: its entry points are recorded)."""
import pytest
import torch

I32, BF, Z = torch.int32, torch.bfloat16, torch.zeros


@pytest.fixture
def b(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as b
    seen = {}

    def record(name, at):
        def call(*a):
            seen.setdefault(name, []).append(a[at])
            return 0
        monkeypatch.setattr(b, name, call)

    record("_adapters", -2)
    record("_adapters_grad", -2)
    record("_route_groups", 0)
    record("_route_groups_grad", -2)
    monkeypatch.setattr(b, "_on", lambda *a, **k: None)
    monkeypatch.setattr(b, "_current_device", lambda: -1)
    monkeypatch.setattr(b, "_here", lambda *a: 0)
    b.seen = seen
    return b


@pytest.mark.parametrize("given", [False, True])
def test_status_pointers(b, given):
    st = Z(1, dtype=I32) if given else None
    x, a, w = (Z(4, 64, dtype=BF, requires_grad=True), Z(2, 8, 64, dtype=BF, requires_grad=True), Z(2, 8, 48, dtype=BF, requires_grad=True))
    out = b.AdapterAdd.apply(x, a, w, Z(2), Z(4, dtype=I32), None, None, st)
    out.sum().backward()
    _, rw = b.RouteGroups.apply(Z(4, 16, requires_grad=True), 2, 1, 1, None, None, False, False, True, 1.0, st)
    rw.sum().backward()
    want = [st.data_ptr() if given else None]
    assert b.seen["_adapters"] == want and b.seen["_adapters_grad"] == want and b.seen["_route_groups_grad"] == want


def test_refusals(b):
    a, w, x = Z(2, 8, 64, dtype=BF), Z(2, 8, 48, dtype=BF), Z(4, 64, dtype=BF)
    for bad in (Z(1), Z(0, dtype=I32), Z(1, dtype=torch.int64), Z(1, dtype=I32, device="meta")):
        with pytest.raises(ValueError, match="dev_status"):
            b.Adapters(a, w, Z(2), bad)
        with pytest.raises(ValueError, match="dev_status"):
            b.AdapterAdd.apply(x, a, w, Z(2), Z(4, dtype=I32), None, None, bad)
        with pytest.raises(ValueError, match="dev_status"):
            b.RouteGroups.apply(Z(4, 16), 2, 1, 1, None, None, False, False, True, 1.0, bad)
