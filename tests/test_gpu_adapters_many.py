"""Batches of very many sequences: the same results, and a cost that grows with their number and no faster."""
import numpy as np
import pytest
import torch

from tests.test_gpu_adapters import DEV, I32, case, check, normal

pytestmark = pytest.mark.gpu


def test_results():
    r = np.random.default_rng(3)
    check(6000, 64, 72, 8, 3, 1, lengths=r.multinomial(6000, np.ones(2500) / 2500).tolist())
    check(9000, 64, 72, 8, 3, 2, lengths=[0] * 3000 + [8990, 10] + [0] * 3000)
    for n in (29, 30, 31, 32, 33, 61, 62, 63, 64, 960, 1021, 1022, 1023, 1024, 1025, 1056, 1057):  # ends of the search's rounds
        lengths = r.multinomial(3000, np.ones(n) / n)
        check(3000, 64, 72, 8, 2, n, lengths=lengths.tolist(), grads=n % 3 == 0)
        lengths[:] = 0
        lengths[[0, n // 2, n - 1]] = 500, 33, 400
        check(940, 64, 72, 8, 2, n, lengths=lengths.tolist(), lead=5 if n % 2 else 0, grads=False)


def test_a_bad_sequence_anywhere_is_flagged():
    import expert_slot_cache_gb300 as M
    x, a, b, scale, ids, starts = case(3000, 64, 72, 8, 2, 1, [6] * 500, none=0.0)
    op = M.Adapters(a, b, scale)
    for at in (0, 31, 32, 250, 498, 499):
        keep = int(ids[at])
        ids[at] = 2
        op.forward(x, ids, None, starts)
        assert int(op.dev_status.item()) == 1
        op.dev_status.zero_()
        ids[at] = keep
        if at:
            s = starts.clone()
            s[at] = s[at + 1] + 1
            op.forward(x, ids, None, s)
            assert int(op.dev_status.item()) == 4
            op.dev_status.zero_()


def test_cost_is_linear():
    """Four times the rows and sequences: about four times the time (16 where every tile walks through all sequences)."""
    import expert_slot_cache_gb300 as M
    took = []
    for n in (8192, 32768):
        x, a, b, scale, ids, starts = case(8 * n, 64, 64, 8, 2, 1, [8] * n, none=0.0)
        op = M.Adapters(a, b, scale)
        out = torch.empty(8 * n, 64, dtype=x.dtype, device=DEV)
        best = 1e9
        for _ in range(4):
            s, e = torch.cuda.Event(True), torch.cuda.Event(True)
            s.record()
            op.forward(x, ids, None, starts, out=out)
            e.record()
            torch.cuda.synchronize()
            best = min(best, s.elapsed_time(e))
        took.append(best)
    assert took[1] <= 8 * took[0], took
