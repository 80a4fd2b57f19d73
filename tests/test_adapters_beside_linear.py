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


def test_refused_before_anything_is_written(lin):
    x, ids, starts = Z(4, 64, dtype=BF), Z(2, dtype=I32), Z(3, dtype=I32)
    buf = Z(4 * 64 + 4096, dtype=BF)
    buf = buf[(-buf.data_ptr() % 16) // 2:]
    rows = buf[:256].view(4, 64)
    bad = [dict(adapter_ids=ids[:0], seq_start=starts[:1]),               # no sequence
           dict(x=buf[:64].expand(4, 64)),                                # rows on top of each other
           dict(out=buf.as_strided((4, 64), (56, 1))),
           dict(x=rows, out=rows),                                        # in place
           dict(x=rows, out=buf[64:64 + 256].view(4, 64)),                # over the next rows
           dict(out=buf[4:260].view(4, 64))]                              # not on 16 bytes
    for kw in bad:
        with pytest.raises((ValueError, lin.b.MoeError)):
            lin.forward(**dict(dict(x=x, adapters=lin.op, adapter_ids=ids, seq_start=starts), **kw))
        assert not lin.written, kw
