"""The router's balance loss against its definition in 64 bits, its gradient against the formula and against
differences of the loss.

Tolerances: a probability is an exp (2 units in the last place, plus the rounding of its argument, at most 2^-24
of |logit - max| < 64) over a sum of up to 1024 terms (32 sequential, 5 in a tree): relative 2^-24 * (64 + 37 + 8) <
1e-5 in p, in d and in every term of the gradient p (f - d), whose error is thus at most 1e-5 of p (f + d).  The
loss adds d over the tokens in 64 bits.  bf16 gradients add half a unit in the last place, 2^-8 of the value at
most.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def plain(logits, ids, coef, starts, mask, sigmoid):
    """loss, counts, gradient, and p (f + d) * coef / T_v (the scale of the gradient's terms), fp64 on the CPU."""
    T, E = logits.shape
    k = ids.shape[1]
    l = logits.double().cpu()
    ids = ids.cpu().numpy()
    starts = [0, T] if starts is None else starts.cpu().tolist()
    valid = np.ones(T, bool) if mask is None else mask.cpu().numpy().astype(bool)
    inside = np.zeros(T, bool)
    for a, b in zip(starts, starts[1:]):
        inside[a:b] = True
    total = max(1, int((valid & inside).sum()))
    loss, counts = 0.0, np.zeros((len(starts) - 1, E), np.int32)
    grad, mag = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for s, (a, b) in enumerate(zip(starts, starts[1:])):
        t = np.arange(a, b)[valid[a:b]]
        if not len(t):
            continue
        flat = ids[t].reshape(-1)
        counts[s] = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
        f = torch.from_numpy(counts[s] * (E / (k * len(t))))
        i = torch.from_numpy(t)
        if sigmoid:
            q = torch.nn.functional.logsigmoid(l[i])
            jac = torch.sigmoid(-l[i])
        else:
            q, jac = l[i], torch.ones_like(l[i])
        p = torch.softmax(q, 1)
        p[torch.isneginf(l[i]).all(1)] = 0  # a row of -inf has no probabilities; a NaN stays a NaN
        d = p @ f
        loss += coef / total * float(d.sum())
        grad[i] = coef / total * p * (f - d[:, None]) * jac
        mag[i] = coef / total * p * (f + d[:, None]) * jac
    return loss, counts, grad, mag


def draw(T, E, k, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = (torch.randn(T, E, generator=g, device=DEV) * spread).to(dtype)
    return logits, torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)


def check(logits, ids, coef=0.01, starts=None, mask=None, sigmoid=False):
    import expert_slot_cache_gb300 as M
    loss, counts, grad, mag = plain(logits, ids, coef, starts, mask, sigmoid)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = M.balance_loss(logits, ids, coef, starts, mask, sigmoid, with_grad=True, dev_status=st)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    assert abs(float(r.loss) - loss) <= 1e-5 * abs(loss) or (np.isnan(loss) and bool(r.loss.isnan())), (float(r.loss), loss)
    tol = 1e-5 * mag + 1e-38
    if logits.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * grad.abs()
    got = r.grad.double().cpu()
    assert torch.equal(got.isnan(), grad.isnan())
    err = (got - grad).abs()[~grad.isnan()]
    assert bool((err <= tol[~grad.isnan()]).all()), float((err / tol[~grad.isnan()]).max())
    again = M.balance_loss(logits, ids, coef, starts, mask, sigmoid, with_grad=True)
    bits = lambda v: v.view(torch.int16 if v.dtype == torch.bfloat16 else torch.int32)  # noqa: E731
    assert torch.equal(bits(r.loss), bits(again.loss)) and torch.equal(bits(r.grad), bits(again.grad))
    only = M.balance_loss(logits, ids, coef, starts, mask, sigmoid)
    assert only.grad is None and torch.equal(bits(only.loss), bits(r.loss)) and torch.equal(only.counts, r.counts)
    return r, int(st.item())


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (2, 9, 9), (7, 33, 2), (64, 128, 8), (255, 61, 4),
                                   (1000, 288, 8), (513, 512, 10), (300, 1024, 16), (4099, 130, 6), (20000, 16, 2)])
def test_one_sequence(T, E, k, dtype, sigmoid):
    logits, ids = draw(T, E, k, T + E, dtype)
    _, st = check(logits, ids, sigmoid=sigmoid)
    assert st == 0


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E,k,n,share", [(50, 16, 2, 50, 0.0), (100, 64, 4, 7, 0.3), (3000, 288, 8, 41, 0.1),
                                           (9000, 128, 8, 3, 0.9), (40, 24, 3, 200, 0.2)])
def test_packed_sequences_and_padding(T, E, k, n, share, sigmoid):
    """Ragged sequences, some of them empty, padded tokens that hold NaN logits and ids out of range."""
    logits, ids = draw(T, E, k, T + n)
    r = np.random.default_rng(n)
    starts = np.concatenate([[0], np.sort(r.integers(0, T + 1, n - 1)), [T]]).astype(np.int32)
    mask = torch.from_numpy(r.random(T) >= share).to(DEV)
    a, b = int(starts[n // 2]), int(starts[n // 2 + 1])
    mask[a:b] = False  # one sequence is padding only
    logits[~mask] = float("nan")
    ids[~mask] = -7
    res, st = check(logits, ids, starts=torch.from_numpy(starts).to(DEV), mask=mask, sigmoid=sigmoid)
    assert st == 0 and not bool(res.grad[~mask].any())
    res2, _ = check(logits, ids, starts=torch.from_numpy(starts).to(DEV), mask=mask.to(torch.uint8), sigmoid=sigmoid)
    assert torch.equal(res.grad, res2.grad)


def test_nothing_valid():
    logits, ids = draw(33, 20, 3, 1)
    res, _ = check(logits, ids, mask=torch.zeros(33, dtype=torch.bool, device=DEV))
    assert float(res.loss) == 0 and not bool(res.grad.any()) and not bool(res.counts.any())


def test_tokens_outside_every_sequence():
    logits, ids = draw(90, 40, 4, 2)
    starts = torch.tensor([10, 30, 30, 75], dtype=torch.int32, device=DEV)
    res, _ = check(logits, ids, starts=starts)
    assert not bool(res.grad[:10].any()) and not bool(res.grad[75:].any())


@pytest.mark.parametrize("sigmoid", [False, True])
def test_extreme_logits(sigmoid):
    """Hard-masked experts (-inf), a row of -inf, and logits whose exponentials leave the fp32 range."""
    logits, ids = draw(40, 48, 4, 3)
    logits[:, 5] = float("-inf")
    logits[4] = float("-inf")
    logits[6] = logits[6] * 0 + 300
    logits[7] = logits[7] * 0 - 300
    logits[7, 3] = -280
    logits[8, 2] = 200.0
    if sigmoid:  # softmax of log-sigmoids: |logit| counts, not |logit - max|
        logits[8, 2] = 60.0
    check(logits, ids, sigmoid=sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_flat_rows_far_from_zero(sigmoid):
    logits, ids = draw(40, 48, 4, 3)
    logits[:, 5] = float("-inf")
    logits[4] = float("-inf")
    logits[6] = 300
    logits[7] = -300
    logits[7, 3] = -280
    logits[9, 4:] = float("-inf")
    res, _ = check(logits, ids, sigmoid=sigmoid)
    assert bool(res.loss.isfinite()) and bool(res.grad.isfinite().all())


def test_nan_row_is_not_hidden():
    import expert_slot_cache_gb300 as M
    logits, ids = draw(9, 20, 2, 4)
    logits[3, 1] = float("nan")
    r = M.balance_loss(logits, ids, 0.1, with_grad=True)
    assert bool(r.loss.isnan()) and bool(r.grad[3].isnan().all()) and bool(r.grad[[0, 1, 2, 4, 5, 6, 7, 8]].isfinite().all())


def test_bad_ids_are_flagged_and_not_counted():
    logits, ids = draw(50, 32, 4, 5)
    ids[7, 1] = 32
    ids[9, 0] = -1
    _, st = check(logits, ids)
    assert st == 1


def test_descending_starts_are_flagged():
    import expert_slot_cache_gb300 as M
    logits, ids = draw(50, 32, 4, 5)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.balance_loss(logits, ids, 0.1, torch.tensor([0, 40, 20, 999], dtype=torch.int32, device=DEV), dev_status=st)
    assert int(st.item()) == 4


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradient_against_differences(sigmoid):
    """Along random directions: (L(l + h v) - L(l - h v)) / 2h of the fp64 loss, f held (the counts do not move)."""
    import expert_slot_cache_gb300 as M
    logits, ids = draw(60, 40, 4, 8)
    starts = torch.tensor([0, 11, 11, 60], dtype=torch.int32, device=DEV)
    r = M.balance_loss(logits, ids, 1.0, starts, sigmoid=sigmoid, with_grad=True)
    rng = np.random.default_rng(0)
    for _ in range(4):
        v = torch.from_numpy(rng.standard_normal((60, 40)))
        h = 1e-5
        up = plain(logits.double().cpu() + h * v, ids, 1.0, starts, None, sigmoid)[0]
        dn = plain(logits.double().cpu() - h * v, ids, 1.0, starts, None, sigmoid)[0]
        got = float((r.grad.double().cpu() * v).sum())
        scale = float((r.grad.double().cpu().abs() * v.abs()).sum())
        # truncation h^2, cancellation 2^-53 / h, and 1e-5 of the gradient's terms
        assert abs(got - (up - dn) / (2 * h)) <= 2e-5 * scale + 1e-9


def test_autograd():
    """loss and gradient through autograd, with the loss scaled on its way."""
    import expert_slot_cache_gb300 as M
    logits, ids = draw(70, 24, 2, 9)
    mask = torch.ones(70, dtype=torch.bool, device=DEV)
    mask[60:] = False
    leaf = logits.clone().requires_grad_(True)
    loss, counts = M.BalanceLoss.apply(leaf * 2.0, ids, 0.5, None, mask, False)
    (loss * 3.0).backward()
    want_loss, want_counts, want, mag = plain(logits * 2.0, ids, 0.5, None, mask, False)
    assert abs(float(loss.detach()) - want_loss) <= 1e-5 * want_loss and np.array_equal(counts.cpu().numpy(), want_counts)
    assert bool(((leaf.grad.double().cpu() - 6 * want).abs() <= 6e-5 * mag + 1e-12).all())


def test_other_streams():
    import expert_slot_cache_gb300 as M
    logits, ids = draw(5000, 128, 8, 10)
    first = M.balance_loss(logits, ids, 0.01, with_grad=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = M.balance_loss(logits, ids, 0.01, with_grad=True)
    torch.cuda.synchronize()
    assert torch.equal(first.grad, r.grad) and torch.equal(first.loss, r.loss)
