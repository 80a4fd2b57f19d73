"""The balance loss where fp32 runs short: logits far from zero with small gradient scales.

The tolerance is that of the ordinary rows (test_gpu_balance): 1e-5 of p (f + d) times the gradient's scale.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_balance import DEV, draw, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1.0, 1e-9, 1e-20])
@pytest.mark.parametrize("shift", [-62, -12, 20, 55, 62])
def test_small_gradients_of_rows_far_from_zero(shift, scale, dtype, sigmoid):
    import expert_slot_cache_gb300 as M
    logits, ids = draw(700, 64, 4, 3)
    logits = (logits + shift).to(dtype)
    _, _, grad, mag = plain(logits, ids, 0.01, None, None, sigmoid)
    r = M.balance_loss(logits, ids, 0.01, sigmoid=sigmoid, with_grad=True, grad_loss=torch.tensor([scale], device=DEV))
    s = float(np.float32(scale))
    tol = s * (1e-5 * mag + (2.0 ** -8 * grad.abs() if dtype == torch.bfloat16 else 0)) + 1e-38
    err = (r.grad.double().cpu() - s * grad).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
