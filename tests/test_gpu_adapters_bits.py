"""The bits that the adapters' sums keep: v whole in its product, no drift where there are many features."""
import pytest
import torch

from tests.test_gpu_adapters import check

pytestmark = pytest.mark.gpu
DEV, BF, I32 = "cuda", torch.bfloat16, torch.int32


def two_ranks(T, n, m, low):
    """x [T][n], a [2][n], b [2][m] with x a_0 = 1 + 2^-9 + low, x a_1 = 1 + 2^-9, b_0 = 1, b_1 = -1."""
    x, a, b = torch.zeros(T, n, dtype=BF, device=DEV), torch.zeros(1, 2, n, dtype=BF, device=DEV), torch.ones(1, 2, m, dtype=BF, device=DEV)
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 2.0 ** -9, low
    a[0, 0, :3] = 1.0
    a[0, 1, :2] = 1.0
    b[0, 1] = -1.0
    return x, a, b


@pytest.mark.parametrize("low", [2.0 ** -14, 2.0 ** -18, 2.0 ** -20])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T", [1, 40, 300, 2000])
def test_differences_of_close_values(T, dtype, low):
    """out = low, exactly: v is held in fp32 (24 bits) and its product is with all of them."""
    import expert_slot_cache_gb300 as M
    x, a, b = two_ranks(T, 136, 72, low)
    ids, starts = torch.zeros(1, dtype=I32, device=DEV), torch.tensor([0, T], dtype=I32, device=DEV)
    one = torch.ones(1, device=DEV)
    op = M.Adapters(a, b, one)
    kept = torch.empty(T, 2, device=DEV)
    assert bool((op.forward(x, ids, None, starts, out_dtype=dtype, kept=kept) == low).all())
    if dtype == BF:  # dx is the same with A and B exchanged
        rev = M.Adapters(b, a, one)
        assert bool((rev.grad(x, None, None, ids, None, starts, with_weights=False).dx == low).all())


@pytest.mark.parametrize("R", [3, 64, 80, 128])
def test_sums_over_many_features_do_not_drift(R):
    """A truncated addition takes less than 2^-23 of the sum, always downwards; one that rounds has no direction.  With at
    most 16 truncated ones in a row the mean of (v - exact) / exact over many sums of positive terms is within
    16 * 2^-23 of 0, however many features there are."""
    import expert_slot_cache_gb300 as M
    T, K = 200, 131072
    g = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.rand(T, K, generator=g, device=DEV) + 0.5).to(BF)
    a = (torch.rand(1, R, K, generator=g, device=DEV) + 0.5).to(BF)
    b = torch.zeros(1, R, 16, dtype=BF, device=DEV)
    op = M.Adapters(a, b, torch.ones(1, device=DEV))
    kept = torch.empty(T, R, device=DEV)
    op.forward(x, torch.zeros(1, dtype=I32, device=DEV), None, torch.tensor([0, T], dtype=I32, device=DEV), kept=kept)
    v = x.double() @ a[0].double().T
    mean = float(((kept.double() - v) / v).mean())
    assert abs(mean) <= 16 * 2.0 ** -23, mean


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T,K,N,R", [(70, 20008, 72, 20), (300, 8264, 9000, 70), (1500, 4160, 264, 128), (5000, 2120, 136, 33), (2500, 131072, 8, 16),
                                     (33, 40000, 40000, 100)])
def test_sums_taken_over(T, K, N, R, dtype):
    """More than 1024 features a CTA, in clusters and tiles of every size; both passes, rows of two sequences."""
    check(T, K, N, R, 2, T + R, lengths=[T - 21, 21], dtype=dtype, none=0.0)
