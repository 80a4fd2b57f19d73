"""Picks of 64-bit arithmetic where exact duplicates stand beside a near neighbour at the k-th place."""
import numpy as np
import pytest
import torch

from tests.test_gpu_groups import DEV, check

pytestmark = pytest.mark.gpu


def neighbours(T, E, copies, sigmoid, seed):
    """Logits and a bias: `copies` experts of one logit and bias, and one expert (the first or the last of all) whose score
    in 64 bits is within some 1e-7 of theirs, now above, now below; the others are far below."""
    r = np.random.default_rng(seed)
    z = (r.normal(size=(T, E)) * 1.5).astype(np.float32)
    bias = np.full(E, -3.0, np.float32)
    at = 1 + r.permutation(E - 2)[:copies]
    lone = 0 if seed % 2 else E - 1
    bias[at], bias[lone] = np.float32(-0.90886205), np.float32(-0.94229984)
    la = r.uniform(2.0, 4.0, T).astype(np.float32)
    z[:, at] = la[:, None]
    gap = float(bias[at[0]]) - float(bias[lone])
    if sigmoid:
        s = 1 / (1 + np.exp(-la.astype(np.float64))) + gap
        ok = s < 0.9999
        s = np.where(ok, s, 0.75)
        ld = np.log(s / (1 - s))
    else:
        z[:, lone] = -np.inf
        e = np.exp(la.astype(np.float64))
        rest = np.exp(z.astype(np.float64)).sum(1)
        ld = np.log((e + gap * rest) / (1 - gap))  # u / (rest + u) - e / (rest + u) = gap
    ulps = r.integers(-3, 4, T).astype(np.int32)
    z[:, lone] = (ld.astype(np.float32).view(np.int32) + ulps).view(np.float32)
    return torch.from_numpy(z).to(DEV), torch.from_numpy(bias).to(DEV)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,copies,k", [(16, 2, 1), (32, 3, 2), (64, 5, 1), (64, 5, 4), (64, 20, 16), (64, 40, 7), (128, 3, 1), (512, 2, 1), (250, 4, 2)])
def test_duplicates_across_the_last_place(E, copies, k, sigmoid):
    for seed in (1, 2):
        logits, bias = neighbours(1500, E, copies, sigmoid, seed)
        check(logits, k, bias=bias, sigmoid=sigmoid)
        if E % 4 == 0:
            check(logits, k, bias=bias, sigmoid=sigmoid, n_group=4, topk_group=3)
