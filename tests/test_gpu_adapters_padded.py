"""Starts padded with empty sequences, as a captured graph's are: the same gradients, at about the same cost; adapters of long
and of short sequences in one batch."""
import pytest
import torch

from tests.test_gpu_adapters import DEV, I32, case, check, normal
from tests.test_gpu_adapters_descending import took

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,R,L,lengths", [
    (4000, 264, 136, 24, 2, [1990, 2010] + [0] * 700),
    (700, 64, 72, 8, 3, [0] * 60 + [300, 0, 395, 5] + [0] * 30),
    (256, 64, 72, 16, 2, [256] + [0] * 40),
    (255, 64, 72, 16, 2, [255] + [0] * 40),
    (2600, 136, 264, 40, 4, [1] * 100 + [1000, 900] + [4] * 150),
    (3000, 64, 72, 100, 5, [3] * 400 + [600, 15, 16, 17, 31] + [0] * 300 + [8] * 140 + [1]),
    (600, 72, 64, 8, 40, [15] * 20 + [16] * 18 + [12] + [0] * 9),
])
def test_padded_and_mixed(T, K, N, R, L, lengths):
    check(T, K, N, R, L, T, lengths=lengths, none=0.0, lead=0)
    check(T + 9, K, N, R, L, T + 1, lengths=lengths, none=0.2, lead=4)


def test_one_adapter_of_each_kind():
    """Adapter 0 has long sequences, 1 short ones, 2 none, 3 exactly 16 rows a sequence, 4 one row fewer."""
    import expert_slot_cache_gb300 as M
    lengths, ids = [], []
    for q in range(60):
        lengths += [70, 3, 0, 16, 16 if q else 15]
        ids += [0, 1, 2, 3, 4]
    lengths += [0] * 1500
    ids += [2] * 1500
    T = sum(lengths)
    x, a, b, scale, _, starts = case(T, 264, 136, 20, 5, 3, lengths)
    ids = torch.tensor(ids, dtype=I32, device=DEV)
    dy = normal(T, 136, g=torch.Generator(device=DEV).manual_seed(4))
    op, kept = M.Adapters(a, b, scale), torch.empty(T, 20, device=DEV)
    op.forward(x, ids, None, starts, kept=kept)
    r = op.grad(dy, x, kept, ids, None, starts)
    s = starts.tolist()
    for l in range(5):
        rows = torch.tensor([t for q in range(len(ids)) if int(ids[q]) == l for t in range(s[q], s[q + 1])] if l != 2 else [], dtype=torch.long, device=DEV)
        want = kept[rows].double().T @ dy[rows].double()
        size = kept[rows].double().abs().T @ dy[rows].double().abs()
        assert bool(((r.db[l].double() - want).abs() <= (len(rows) + 2) * 2.0 ** -23 * size).all()), l
        if l == 2:
            assert not bool(r.da[l].any())
    again = op.grad(dy, x, kept, ids, None, starts)
    assert torch.equal(r.da, again.da) and torch.equal(r.db, again.db) and int(op.dev_status.item()) == 0


def test_padding_costs_little():
    import expert_slot_cache_gb300 as M
    times = []
    for n in (2, 1024):
        x, a, b, scale, ids, starts = case(8192, 512, 512, 32, 2, 1, [4000, 4192] + [0] * (n - 2), none=0.0)
        op, kept = M.Adapters(a, b, scale), torch.empty(8192, 32, device=DEV)
        dy = normal(8192, 512, g=torch.Generator(device=DEV).manual_seed(1))
        op.forward(x, ids, None, starts, kept=kept)
        times.append(took(lambda: op.grad(dy, x, kept, ids, None, starts)))
    assert times[1] <= 4 * times[0], times  # (20 times where empty sequences counted)


def test_captured_with_other_starts():
    """One graph, replayed with other lengths: the choice is the device's."""
    import expert_slot_cache_gb300 as M
    T, n = 1200, 300
    x, a, b, scale, ids, starts = case(T, 72, 64, 8, 2, 1, [4] * n, none=0.0)
    dy, kept, op = normal(T, 64, g=torch.Generator(device=DEV).manual_seed(1)), torch.empty(T, 8, device=DEV), M.Adapters(a, b, scale)

    def step():
        out = op.forward(x, ids, None, starts, kept=kept)
        return [out, *op.grad(dy, x, kept, ids, None, starts)]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for lengths in ([4] * n, [600, 600] + [0] * (n - 2), [0] * 100 + [1] * 100 + [1100] + [0] * 99):
        starts.copy_(torch.tensor([0] + lengths, dtype=I32, device=DEV).cumsum(0).to(I32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(p, q) for p, q in zip(got, step()))
