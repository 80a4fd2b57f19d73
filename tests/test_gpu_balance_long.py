"""The balance loss of a batch of many tokens: d is added in 64 bits.

Every token has the same three logits, so that each of its d has the same error and roundings of the sum would add up.
Tolerance: ex2.approx 2^-22, its argument (below 2) 2^-25, twice (numerator and sum); adds, products, reciprocal and f
nine more roundings of 2^-24: 2^-21 + 2^-24 + 9 * 2^-24 < 1.1e-6.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("row", [(0.7, -0.5, -0.9), (0.3, 0.2, -1.1)])
def test_the_same_row_many_times(row):
    import expert_slot_cache_gb300 as M
    T = 1 << 24
    logits = torch.tensor(row, device=DEV).repeat(T, 1)
    ids = (torch.arange(T, device=DEV, dtype=torch.int32) % 8 > 5).to(torch.int32)[:, None].contiguous()
    r = M.balance_loss(logits, ids, 1.0)
    assert r.counts.tolist() == [[3 * T // 4, T // 4, 0]]
    p = torch.softmax(logits[0].double(), 0)
    want = float(3 * (0.75 * p[0] + 0.25 * p[1]))
    assert abs(float(r.loss) - want) <= 1.1e-6 * want, (float(r.loss), want)
