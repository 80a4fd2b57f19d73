"""NaN and +inf among the logits: what the scores are then by definition, and no other token's picks change."""
import pytest
import torch

from tests.test_gpu_groups import DEV, check, draw, steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,g,k", [(48, 6, 3, 6), (128, 8, 3, 8), (512, 8, 4, 10), (100, 1, 1, 5), (32, 32, 4, 4)])
def test_rows_with_nan_and_infinity(E, G, g, k, dtype, sigmoid, renormalise):
    import expert_slot_cache_gb300 as M
    clean = draw(60, E, E, dtype)
    logits = clean.clone()
    logits[3, 5] = float("nan")
    logits[10, E - 1] = float("nan")
    logits[11, ::2] = float("nan")
    logits[12] = float("nan")
    logits[20, 7] = float("inf")
    logits[21, [1, E - 2]] = float("inf")
    logits[30, 4], logits[30, 9] = float("nan"), float("inf")
    ok = ~(logits.isnan() | logits.isinf()).any(1)
    for bias in (None, steps(E, 2)):
        for group_max in (False, True):
            kw = dict(n_group=G, topk_group=g, sigmoid=sigmoid, group_max=group_max, renormalise=renormalise)
            r = check(logits, k, bias=bias, **kw)
            c = M.route_groups(clean, k, sel_bias=bias, **kw)
            assert torch.equal(r.ids[ok], c.ids[ok]) and torch.equal(r.w[ok], c.w[ok])
