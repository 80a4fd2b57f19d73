"""A call that is given a stream allocates for it: what it takes from the allocator belongs to the stream that its
kernels run on (no GPU: the library's entry points, the stream context and the allocations are recorded)."""
import contextlib

import pytest
import torch

I32 = torch.int32


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

    for name in ("_route", "_permute", "_ffn", "_ffn_q8", "_ffn_w4", "_balance", "_w4_pack", "_w4_linear", "_experts_w4"):
        monkeypatch.setattr(b, name, lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(b, "_on", lambda *a, **k: None)
    monkeypatch.setattr(b, "_current", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(b, "_current_device", lambda: -1)
    monkeypatch.setattr(b, "_here", lambda *a: 0)
    b.seen = seen
    lin = b.W4Linear(torch.zeros(b.w4_bytes(64, 16, 64), dtype=torch.uint8), 64, 16, 64, max_tokens=2)
    ex = b.W4Experts(torch.zeros(16, b.w4_slab_bytes(256, 128, 64), dtype=torch.uint8), 256, 128, 2, 16, 64, max_tokens=2)
    x, ids, lst = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=I32), [torch.zeros(17, dtype=I32)] * 4
    codes, scales = torch.zeros(64, 16, dtype=torch.uint8), torch.zeros(1, 16, dtype=torch.bfloat16)
    logits, wr, w, s = torch.zeros(2, 16), torch.zeros(256, 16), torch.zeros(2, 2), Stream()
    b.calls = dict(
        balance=lambda: b.balance_loss(logits, ids, 0.1, with_grad=True, stream=s),
        ffn_w4=lambda: b.expert_ffn_w4(x, 2, 128, 16, 64, *lst, 16, ex.pool, stream=s),
        ffn_q8=lambda: b.expert_ffn_q8(x, 2, 128, 16, *lst, 16, ex.pool, stream=s),
        ffn=lambda: b.expert_ffn(x, 2, 128, 16, *lst, 16, ex.pool, stream=s),
        route=lambda: b.route(x, wr, 2, stream=s),
        permute=lambda: b.permute(ids, 16, None, s),  # by position
        pack=lambda: b.w4_pack(codes, scales, 64, stream=s),
        linear=lambda: lin.forward(x[:, :64], stream=s),
        experts=lambda: ex.forward(x, ids, w, stream=s))
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    return b


@pytest.mark.parametrize("call", ["balance", "ffn_w4", "ffn_q8", "ffn", "route", "permute", "pack", "linear", "experts"])
def test_allocations_belong_to_the_stream(b, call):
    b.calls[call]()
    assert b.seen and all(b.seen)


@pytest.mark.gpu
def test_a_busy_stream_beside_the_current_one():
    """Kernels queued behind a long wait on their stream; the current stream takes and overwrites memory meanwhile."""
    import expert_slot_cache_gb300 as M
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(1)
    logits = torch.randn(5000, 128, generator=g, device=dev)
    ids = torch.topk(logits, 8, dim=1).indices.to(I32)
    want = M.balance_loss(logits, ids, 0.01, with_grad=True)
    busy = torch.randn(6000, 6000, generator=g, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            busy = busy @ busy * 1e-3
    got = M.balance_loss(logits, ids, 0.01, with_grad=True, stream=s)
    fill = [torch.full((n,), 255, dtype=torch.uint8, device=dev) for n in (512, 20480, 40960, 131072, 1 << 20, 1 << 22)]
    torch.cuda.synchronize()
    assert torch.equal(want.loss, got.loss) and torch.equal(want.grad, got.grad) and torch.equal(want.counts, got.counts)
    assert all(bool((f == 255).all()) for f in fill)
