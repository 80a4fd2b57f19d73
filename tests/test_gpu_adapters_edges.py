"""The adapters at the ends of their ranges, and calls that overlap."""
import pytest
import torch

from tests.test_gpu_adapters import BF, DEV, I32, case, check, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,R,L,lengths", [(3, 131072, 8, 1, 1, None), (200, 131072, 16, 3, 1, [200]), (2, 8, 131072, 128, 1, None),
                                               (90, 16, 131072, 5, 2, [40, 50]), (64, 8, 8, 1, 65535, None), (300, 8, 16, 2, 65535, [100, 200])])
def test_largest_sizes(T, K, N, R, L, lengths):
    check(T, K, N, R, L, T + R, lengths=lengths, none=0.0)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("R", [15, 16, 17, 31, 48, 63, 65, 79, 81, 95, 96, 112, 127])
def test_ranks(R, dtype):
    """Every size of the rings and of the columns of the weights' gradients."""
    check(333, 200, 328, R, 2, R, lengths=[130, 1, 202], dtype=dtype, none=0.0)


def test_far_more_sequences_than_rows():
    check(200, 64, 72, 8, 3, 1, lengths=[0] * 3000 + [150] + [0] * 2000 + [50] + [0] * 500, none=0.0)
    check(3, 64, 72, 8, 3, 2, lengths=[0] * 500 + [2] + [0] * 300, none=0.0, lead=1)


def test_short_and_long_sequences_in_every_order():
    for k, lengths in enumerate(([4, 5, 4, 60, 1], [1, 2, 3, 4, 5, 6], [500] + [1] * 30, [1] * 30 + [500], [4] * 20 + [33] * 3 + [4] * 20)):
        check(sum(lengths) + 11, 136, 264, 20, 4, k, lengths=lengths, lead=5)


def test_two_streams_at_once():
    """Calls of one handle on two streams: nothing is shared but the weights and the status."""
    import expert_slot_cache_gb300 as M
    args = [case(2000, 256, 520, 24, 3, seed, [700, 3, 1297], none=0.0) for seed in (1, 2)]
    a, b, scale = args[0][1:4]
    op = M.Adapters(a, b, scale)
    g = torch.Generator(device=DEV).manual_seed(4)
    dy, kept = [normal(2000, 520, g=g) for _ in range(2)], [torch.empty(2000, 24, device=DEV) for _ in range(2)]

    def step(i, stream=None):
        x, ids, starts = args[i][0], args[i][4], args[i][5]
        out = op.forward(x, ids, None, starts, kept=kept[i], stream=stream)
        return [out, *op.grad(dy[i], x, kept[i], ids, None, starts, stream=stream)]

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(step(i, streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for r in got[i] for p, q in zip(r, want[i]))
    assert int(op.dev_status.item()) == 0


def test_weights_are_read_where_they_are():
    import expert_slot_cache_gb300 as M
    for T, lengths in ((4, None), (300, [300])):
        x, a, b, scale, ids, starts = case(T, 64, 72, 8, 2, 5, lengths, none=0.0)
        op = M.Adapters(a, b, scale)
        first = op.forward(x, ids, None, starts)
        a.mul_(2)
        scale.mul_(0.5)
        assert torch.equal(op.forward(x, ids, None, starts), first)  # powers of two: exactly the same
        b.zero_()
        assert not bool(op.forward(x, ids, None, starts).any())


def test_the_same_adapter_and_rows_of_a_larger_buffer():
    """Views into larger buffers: what is beside them stays as it is."""
    import expert_slot_cache_gb300 as M
    x, a, b, scale, ids, starts = case(260, 64, 72, 8, 1, 5, [200, 60], none=0.0)
    op = M.Adapters(a, b, scale)
    buf = torch.full((300, 72), 3.0, dtype=BF, device=DEV)
    base = torch.zeros(260, 72, dtype=BF, device=DEV)
    out = op.forward(x, ids, base, starts, out=buf[20:280])
    assert torch.equal(out, op.forward(x, ids, base, starts))
    assert bool((buf[:20] == 3).all()) and bool((buf[280:] == 3).all())
    assert torch.equal(op.forward(x, torch.zeros(1, dtype=I32, device=DEV), base, torch.tensor([0, 260], dtype=I32, device=DEV)).float().sign(), out.float().sign())
