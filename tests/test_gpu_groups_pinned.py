"""Selection biases of +inf: a pinned expert is picked, and its group with it."""
import pytest
import torch

from tests.test_gpu_groups import DEV, check, draw, steps

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,g,k", [(48, 4, 2, 6), (128, 8, 3, 8), (512, 8, 4, 10), (512, 16, 2, 8), (16, 16, 3, 3), (1024, 16, 4, 8), (340, 17, 2, 7)])
def test_pinned_experts(E, G, g, k, dtype, sigmoid):
    logits = draw(60, E, E + G, dtype)
    group = E // G
    for pinned in ([E - 1], [0], [E - 1, E - group], [E // 2, E - 1], [group, 2 * group, E - 1, E - group]):
        for rest in (0.0, -INF):  # the others of the pinned groups as they are, or ruled out
            bias = steps(E, 7)
            for e in pinned:
                bias[e // group * group:(e // group + 1) * group] += rest
            bias[pinned] = INF
            left = E - group * len({e // group for e in pinned}) + len(pinned) if rest else E
            for group_max in (False, True):
                if left < E and g * group - group + 1 < k:
                    continue
                r = check(logits, k, n_group=G, topk_group=g, bias=bias, sigmoid=sigmoid, group_max=group_max, scale=2.5)
                if len({e // group for e in pinned}) <= g and len(pinned) <= k:
                    for e in pinned:
                        assert bool((r.ids == e).any(1).all())
    check(logits, k, bias=torch.full((E,), INF, device=DEV), n_group=G, topk_group=g, sigmoid=sigmoid)
