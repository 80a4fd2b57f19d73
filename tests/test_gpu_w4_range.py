"""The 4-bit operators over the whole range of their inputs: outliers, values near the end of fp32's range,
infinities, NaN.

References are fp64 products of the unpacked weights.  The linear layer's tolerance is that of the ordinary sizes,
(K / 32 + 40) fp32 roundings of 2^-23 of the sum of |x w|: it does not grow with an input whose weights are zero.
The experts' is theirs, a relative L2 of 2.4e-3 (bf16 outputs).
"""
import pytest
import torch

from tests._setup import rel_l2
from tests.test_gpu_w4 import RL2_OUT_BF16, check_linear, dequant, draw_experts, draw_routing, draw_w4, experts_plain

pytestmark = pytest.mark.gpu
DEV = "cuda"

# K, N, group, T: weight streams of one, two and four groups of eight rows, and of several tiles a warp; the large tiles
STREAMS = [(520, 100, 64, 1), (520, 100, 32, 5), (264, 70, 128, 16), (520, 100, 64, 24), (128, 80000, 128, 3)]
LARGE = [(2048, 2048, 64, 200), (4096, 1024, 32, 300)]


def make(K, N, group, T, seed, zero_input=None):
    import expert_slot_cache_gb300 as M
    codes, scales = draw_w4(K, N, group, seed)
    if zero_input is not None:
        codes[zero_input] = 8
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16)
    op = M.W4Linear(M.w4_pack(codes.to(DEV), scales.to(DEV), group), K, N, group, max_tokens=T, out_dtype=torch.float32)
    return op, x, dequant(codes, scales, group)


@pytest.mark.parametrize("outlier", [1e4, 1e6])
@pytest.mark.parametrize("K,N,group,T", STREAMS + LARGE)
def test_an_input_without_weights_costs_no_accuracy(K, N, group, T, outlier):
    """One input is far larger than the others and meets zeros in every column."""
    op, x, w = make(K, N, group, T, T, zero_input=37)
    x[:, 37] = outlier
    check_linear(op.forward(x.to(DEV)), x, w, torch.float32)


@pytest.mark.parametrize("K,N,group,T", STREAMS + LARGE)
def test_finite_rows_near_the_end_of_the_range(K, N, group, T):
    """Rows whose results are finite although sums of |x| would not be; a result above the range is an infinity."""
    op, x, w = make(K, N, group, T, T + 3, zero_input=21)
    x[0] *= 2.0 ** 124
    if T > 1 and (K, N, group, T) not in LARGE:  # (the large tiles keep 2^39 between the values of a row)
        x[1, 21] = -3.3e38
    y = op.forward(x.to(DEV)).cpu()
    check_linear(y, x, w, torch.float32)
    x[0] = x[0].sign() * 3e38
    want = x[:1].double() @ w
    far = want.abs() > 3.5e38
    assert bool(far.any()) and torch.equal(op.forward(x.to(DEV)).cpu()[:1][far].double(), want[far].sign() * float("inf"))


@pytest.mark.parametrize("K,N,group,T", STREAMS + LARGE)
def test_infinities_and_nan_give_what_the_formula_gives(K, N, group, T):
    """inf * w is an infinity of w's sign, inf * 0 and inf - inf are NaN; other rows do not notice."""
    op, x, w = make(K, N, group, T, T + 7)
    rows = min(T, 4)
    x[0, 9] = float("inf")
    if rows > 1:
        x[1, K - 1] = float("-inf")
    if rows > 2:
        x[2, 3], x[2, 70] = float("inf"), float("-inf")
    if rows > 3:
        x[3, 0] = float("nan")
    y, want = op.forward(x.to(DEV)).double().cpu(), x.double() @ w
    assert torch.equal(y[:rows].isnan(), want[:rows].isnan())
    assert torch.equal(y[:rows].nan_to_num(0, 1, -1), want[:rows].nan_to_num(0, 1, -1))
    assert not bool(y[:rows].isfinite().any())
    if T > rows:
        check_linear(y[rows:], x[rows:], w, torch.float32)


@pytest.mark.parametrize("outlier", [1e6, 1e30, 3.3e38])
@pytest.mark.parametrize("T", [1, 8, 45])  # streams over the kernel's own groups, and over given ones
def test_experts_with_an_input_without_weights(T, outlier):
    import expert_slot_cache_gb300 as M
    H, I, E, k, group = 320, 96, 70, 13, 64
    codes, scales = draw_experts(H, I, E, group, 2)
    codes[:, : H * I].view(E, H, I)[:, 77] = 8
    codes[:, H * I: 2 * H * I].view(E, H, I)[:, 77] = 8
    op = M.W4Experts(M.w4_pack_slabs(codes, scales, H, I, group), H, I, k, E, group, max_tokens=T)
    x = torch.randn(T, H, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).to(torch.bfloat16)
    x[:, 77] = outlier
    ids, w = draw_routing(T, E, k, T)
    out, want = op.forward(x, ids, w), experts_plain(x, ids, w, codes, scales, H, I, group)
    assert rel_l2(out.double().cpu(), want.cpu()) <= RL2_OUT_BF16
    x[0, 5] = float("inf")  # one token loses its finite values, no other
    out = op.forward(x, ids, w)
    assert not bool(out[0].isfinite().any())
    if T > 1:
        assert rel_l2(out[1:].double().cpu(), want[1:].cpu()) <= RL2_OUT_BF16
