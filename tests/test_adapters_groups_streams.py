"""The adapters' and the group routing's calls that are given a stream allocate for it, and refuse tensors of another
device (no GPU: the library's entry points, the stream context and the allocations are recorded, and the "meta" device
stands for another one)."""
import contextlib

import pytest
import torch

I32, BF, Z = torch.int32, torch.bfloat16, torch.zeros


class Stream:
    cuda_stream = 4711


@pytest.fixture
def b(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as b
    current, seen = [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def recorded(make):
        def alloc(*a, **k):
            seen.append(bool(current))
            return make(*a, **k)
        return alloc

    for name in ("_route_groups", "_route_groups_grad", "_adapters", "_adapters_grad", "_w4_linear"):
        monkeypatch.setattr(b, name, lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(b, "_on", lambda *a, **k: None)
    monkeypatch.setattr(b, "_current_device", lambda: -1)
    monkeypatch.setattr(b, "_here", lambda *a: 0)
    b.seen = seen
    op = b.Adapters(Z(2, 8, 64, dtype=BF), Z(2, 8, 48, dtype=BF), Z(2))
    lin = b.W4Linear(Z(b.w4_bytes(64, 48, 64), dtype=torch.uint8), 64, 48, 64, max_tokens=4)
    x, dy, kept, ids, starts, s = Z(4, 64, dtype=BF), Z(4, 48, dtype=BF), Z(4, 8), Z(2, dtype=I32), Z(3, dtype=I32), Stream()
    b.calls = dict(
        route=lambda: b.route_groups(Z(4, 16), 2, stream=s),
        route_grad=lambda: b.route_groups_grad(Z(4, 16), Z(4, 2, dtype=I32), Z(4, 2), stream=s),
        forward=lambda: op.forward(x, ids, seq_start=starts, stream=s),
        grad=lambda: op.grad(dy, x, kept, ids, seq_start=starts, stream=s),
        linear=lambda: lin.forward(x, adapters=op, adapter_ids=ids, seq_start=starts, stream=s))
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    return b


@pytest.mark.parametrize("call", ["route", "route_grad", "forward", "grad", "linear"])
def test_allocations_belong_to_the_stream(b, call):
    b.calls[call]()
    assert b.seen and all(b.seen)


def test_adapters_of_two_devices():
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300 as M
    with pytest.raises(ValueError, match="on cpu, meta"):
        M.Adapters(Z(2, 8, 64, dtype=BF), Z(2, 8, 48, dtype=BF, device="meta"), Z(2))


@pytest.mark.gpu
def test_host_tensors_beside_device_tensors():
    """Refused on the host: none of these pointers reaches a kernel."""
    import expert_slot_cache_gb300 as M
    dev = "cuda"
    logits = torch.randn(8, 16, device=dev)
    with pytest.raises(ValueError, match="sel_bias"):
        M.route_groups(logits, 2, sel_bias=Z(16))
    with pytest.raises(ValueError, match="token_mask"):
        M.route_groups(logits, 2, token_mask=torch.ones(8, dtype=torch.bool))
    with pytest.raises(ValueError, match="ids"):
        M.route_groups_grad(logits, Z(8, 2, dtype=I32), Z(8, 2, device=dev))
    with pytest.raises(ValueError, match="grad_w"):
        M.route_groups_grad(logits, Z(8, 2, dtype=I32, device=dev), Z(8, 2))
    op = M.Adapters(Z(2, 8, 64, dtype=BF, device=dev), Z(2, 8, 48, dtype=BF, device=dev), Z(2, device=dev))
    x, ids, starts = Z(4, 64, dtype=BF, device=dev), Z(2, dtype=I32, device=dev), torch.tensor([0, 1, 4], dtype=I32, device=dev)
    for name, kw in (("x", dict(x=x.cpu())), ("ids", dict(ids=ids.cpu())), ("seq_start", dict(seq_start=starts.cpu())),
                     ("base", dict(base=Z(4, 48, dtype=BF))), ("out", dict(out=Z(4, 48, dtype=BF))), ("kept", dict(kept=Z(4, 8)))):
        with pytest.raises(ValueError, match=f"{name}: on cpu"):
            op.forward(**dict(dict(x=x, ids=ids, seq_start=starts), **kw))
    dy, kept = Z(4, 48, dtype=BF, device=dev), Z(4, 8, device=dev)
    for name, kw in (("dy", dict(dy=dy.cpu())), ("x", dict(x=x.cpu())), ("kept", dict(kept=kept.cpu())), ("base", dict(base=x.cpu()))):
        with pytest.raises(ValueError, match=f"{name}: on cpu"):
            op.grad(**dict(dict(dy=dy, x=x, kept=kept, ids=ids, seq_start=starts), **kw))
    square = M.Adapters(Z(2, 8, 64, dtype=BF, device=dev), Z(2, 8, 64, dtype=BF, device=dev), Z(2, device=dev))
    with pytest.raises(M.MoeError):
        square.forward(x, ids, seq_start=starts, out=x)  # rows are read while others are written
