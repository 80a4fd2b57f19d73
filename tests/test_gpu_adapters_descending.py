"""Starts that descend are an error that is flagged; what is done until then stays as much as the rows ask for."""
import numpy as np
import pytest
import torch

from tests.test_gpu_adapters import DEV, I32, case, normal

pytestmark = pytest.mark.gpu


def took(call):
    best = 1e9
    for _ in range(4):
        s, e = torch.cuda.Event(True), torch.cuda.Event(True)
        s.record()
        call()
        e.record()
        torch.cuda.synchronize()
        best = min(best, s.elapsed_time(e))
    return best


@pytest.mark.parametrize("T,n", [(2000, 400), (12800, 400), (12800, 200), (2000, 64)])
def test_no_more_work(T, n):
    """Every other sequence as long as the batch: n T / 2 rows in all, of which no more than T are one adapter's work."""
    import expert_slot_cache_gb300 as M
    good = np.linspace(0, T, n + 1).astype(np.int32)
    x, a, b, scale, ids, _ = case(T, 64, 72, 8, 1, 5, [0] * n, none=0.0)
    op = M.Adapters(a, b, scale)
    dy, kept = normal(T, 72, g=torch.Generator(device=DEV).manual_seed(1)), torch.zeros(T, 8, device=DEV)
    back = np.where(np.arange(n + 1) % 2 == 0, 0, T).astype(np.int32)
    times = []
    for starts in (good, back):
        st = torch.from_numpy(starts).to(DEV)
        op.dev_status.zero_()
        times.append(took(lambda: (op.forward(x, ids, None, st, kept=kept), op.grad(dy, x, kept, ids, None, st))))
        assert int(op.dev_status.item()) == (4 if starts is back else 0)
    assert times[1] <= 4 * times[0] + 0.2, times
    # and the next call with good starts is right again
    st = torch.from_numpy(good).to(DEV)
    op.dev_status.zero_()
    op.forward(x, ids, None, st, kept=kept)
    r = op.grad(dy, x, kept, ids, None, st)
    want = kept.double().T @ dy.double()
    size = kept.double().abs().T @ dy.double().abs()
    assert bool(((r.db[0].double() - want).abs() <= (T + 2) * 2.0 ** -23 * size).all()) and int(op.dev_status.item()) == 0
