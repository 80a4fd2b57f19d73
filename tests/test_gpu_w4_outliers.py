"""The routed 4-bit experts where a token has inputs far above the rest whose weights are zero: the results are those of
the rest, on every path, whoever shares the batch.

References are fp64; the tolerances are those of ordinary tokens (test_gpu_w4): relative L2 of 2.4e-3 for bf16 outputs
(twice that for a single token), 2^-11 for the fp32 rows of the large tiles.
"""
import pytest
import torch

from tests._setup import rel_l2
from tests.test_gpu_w4 import RL2_OUT_BF16, RL2_Y_LARGE, draw_experts, draw_routing, experts_plain, ffn_plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
INPUT = 77


def draw(H, I, E, group, seed):
    codes, scales = draw_experts(H, I, E, group, seed)
    codes[:, : H * I].view(E, H, I)[:, INPUT] = 8
    codes[:, H * I: 2 * H * I].view(E, H, I)[:, INPUT] = 8
    return codes, scales


def check(H, I, E, k, T, group, outliers):
    import expert_slot_cache_gb300 as M
    codes, scales = draw(H, I, E, group, T)
    pool = M.w4_pack_slabs(codes, scales, H, I, group)
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T + 7), device=DEV).to(torch.bfloat16)
    x[:, INPUT] = outliers.to(DEV).to(torch.bfloat16)
    ids, w = draw_routing(T, E, k, T, 0.5)
    op = M.W4Experts(pool, H, I, k, E, group, max_tokens=T)
    out = op.forward(x, ids, w)
    assert int(op.dev_status.item()) == 0
    want = experts_plain(x, ids, w, codes, scales, H, I, group)
    assert rel_l2(out.double().cpu(), want.cpu()) <= RL2_OUT_BF16
    worst = ((out.double() - want).norm(dim=1) / want.norm(dim=1)).max()
    assert float(worst) <= 2 * RL2_OUT_BF16, float(worst)
    assert torch.equal(out, op.forward(x, ids, w))
    g = M.permute(ids, E)
    y = M.expert_ffn_w4(x, k, I, E, group, g.offset, g.rows, g.act_e, g.n_act, E, pool)
    rows, flat = g.rows.long(), ids.reshape(-1).long()
    for e in torch.unique(flat).tolist()[:6]:
        p = torch.nonzero(flat[rows] == e).reshape(-1)
        wy = ffn_plain(x[rows[p] // k], codes[e], scales[e], H, I, group)
        worst = ((y[p].double() - wy).norm(dim=1) / wy.norm(dim=1)).max()
        assert float(worst) <= RL2_Y_LARGE, (e, float(worst))


# many rows of an expert; one tile and several, ragged widths, several groups' sizes
LARGE = [(2048, 256, 8, 2, 700, 128), (320, 96, 5, 3, 129, 32), (256, 544, 3, 2, 900, 64)]


@pytest.mark.parametrize("ratio", [3e3, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("H,I,E,k,T,group", LARGE)
def test_every_token(H, I, E, k, T, group, ratio):
    check(H, I, E, k, T, group, torch.full((T,), ratio))


@pytest.mark.parametrize("H,I,E,k,T,group", LARGE)
def test_some_tokens(H, I, E, k, T, group):
    """One token of the batch alone, and tokens of every ratio side by side."""
    one = torch.ones(T)
    one[T // 3] = -1e5
    check(H, I, E, k, T, group, one)
    check(H, I, E, k, T, group, 10.0 ** (torch.arange(T) % 7))


def test_tokens_of_any_size():
    """Whole tokens from 2^-30 to 2^30 of the usual, beside one of zeros: rows have their own powers of two."""
    import expert_slot_cache_gb300 as M
    H, I, E, k, T, group = 256, 128, 4, 2, 244, 64
    codes, scales = draw(H, I, E, group, 3)
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    x = (x * 2.0 ** (torch.arange(T, device=DEV) % 61 - 30)[:, None]).to(torch.bfloat16)
    x[5] = 0
    ids, w = draw_routing(T, E, k, T)
    op = M.W4Experts(M.w4_pack_slabs(codes, scales, H, I, group), H, I, k, E, group, max_tokens=T)
    out, want = op.forward(x, ids, w), experts_plain(x, ids, w, codes, scales, H, I, group)
    assert not bool(out[5].any())
    keep = [t for t in range(T) if t != 5]
    worst = ((out.double() - want).norm(dim=1)[keep] / want.norm(dim=1)[keep]).max()
    assert float(worst) <= 2 * RL2_OUT_BF16, float(worst)
