"""W4Linear's adapters: arguments that would be dropped or refused after the projection has been written (no GPU: the
library's entry points are recorded)."""
import pytest
import torch

I32, BF, Z = torch.int32, torch.bfloat16, torch.zeros


@pytest.fixture
def lin(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as b
    written = []
    monkeypatch.setattr(b, "_w4_linear", lambda *a: written.append(a) or 0)
    monkeypatch.setattr(b, "_on", lambda *a, **k: None)
    monkeypatch.setattr(b, "_current_device", lambda: -1)
    monkeypatch.setattr(b, "_here", lambda *a: 0)
    lin = b.W4Linear(Z(b.w4_bytes(64, 64, 64), dtype=torch.uint8), 64, 64, 64, max_tokens=4)
    lin.written, lin.op, lin.b = written, b.Adapters(Z(2, 8, 64, dtype=BF), Z(2, 8, 64, dtype=BF), Z(2)), b
    return lin


def test_ids_without_adapters(lin):
    x = Z(4, 64, dtype=BF)
    for kw in (dict(adapter_ids=Z(4, dtype=I32)), dict(seq_start=Z(3, dtype=I32)), dict(adapter_ids=Z(2, dtype=I32), seq_start=Z(3, dtype=I32))):
        with pytest.raises(ValueError, match="without adapters"):
            lin.forward(x, **kw)
    assert not lin.written
