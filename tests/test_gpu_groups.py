"""Group-limited routing against its definition in 64 bits, picks exactly; the gradient of its weights against the
formula and against differences.

Tolerances: a score is an exp (2 units in the last place, plus the rounding of its argument, at most 2^-24 of
|logit - max| < 64), a weight that over a sum of up to 1024 of them (32 sequential, 5 in a tree), a product with the
scale: relative 2^-24 * (64 + 37 + 8) < 1e-5.  A gradient is a product of weights and differences g - W, both of which
are off by 1e-5 of their terms' sizes: 2e-5 of s (|g| + sum |g_i| w_i).  bf16 gradients add half a step, 2^-8.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def scores(l, sigmoid):
    if sigmoid:
        return torch.where(l >= 0, 1 / (1 + torch.exp(-l)), torch.exp(l) / (1 + torch.exp(l)))
    return torch.softmax(l, 1)


def plain(logits, k, n_group=1, topk_group=1, bias=None, mask=None, sigmoid=False, group_max=False, renormalise=True,
          scale=1.0):
    """The definition, fp64 on the CPU: picks, weights."""
    l = logits.double().cpu()
    T, E = l.shape
    s = scores(l, sigmoid).numpy()
    l = l.numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    low = lambda v: np.where(np.isnan(v), -1e300, np.maximum(v, -1e290))  # noqa: E731  NaN behind -inf
    for t in range(T):
        if mask is not None and not bool(mask[t]):
            continue
        c = l[t] if b is None else s[t] + b
        pool = np.arange(E)
        if topk_group < n_group:
            by = s[t] if b is None and not group_max else c
            top = -np.sort(-low(by).reshape(n_group, -1), axis=1)
            g = top[:, 0] if group_max or E == n_group else top[:, 0] + top[:, 1]
            stay = np.sort(np.lexsort((np.arange(n_group), -g))[:topk_group])
            pool = (stay[:, None] * (E // n_group) + np.arange(E // n_group)).reshape(-1)
        ids[t] = pool[np.lexsort((pool, -low(c[pool])))[:k]]
        z = l[t][ids[t]]
        if not renormalise:
            w[t] = s[t][ids[t]]
        elif not np.isneginf(z).all():
            q = np.where(z >= 0, 0, z) - np.log1p(np.exp(-np.abs(z))) if sigmoid else z
            q = np.exp(q - q.max())
            w[t] = q / q.sum()
    return ids, w * scale


def draw(T, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(T, E, generator=g, device=DEV) * spread).to(dtype)


def steps(E, seed, size=0.001):
    g = torch.Generator(device=DEV).manual_seed(seed + 99)
    return torch.round(torch.randn(E, generator=g, device=DEV) * 40) * size


def check(logits, k, **kw):
    import expert_slot_cache_gb300 as M
    own = dict(kw)
    own["sel_bias"] = own.pop("bias", None)
    own["token_mask"] = own.pop("mask", None)
    r = M.route_groups(logits, k, **own)
    ids, w = plain(logits, k, **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    got = r.w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(w))
    assert (np.abs(got - w)[~np.isnan(w)] <= 1e-5 * np.abs(w)[~np.isnan(w)] + 1e-37).all()
    again = M.route_groups(logits, k, **own)
    assert torch.equal(r.ids, again.ids) and torch.equal(r.w.view(torch.int32), again.w.view(torch.int32))
    return r


SHAPES = [(1, 1, 1, 1, 1), (1, 128, 8, 8, 4), (3, 6, 2, 6, 5), (2, 9, 9, 1, 1), (5, 32, 4, 32, 4), (7, 33, 2, 3, 2), (64, 512, 10, 16, 4), (65, 24, 6, 2, 1),
          (200, 288, 8, 8, 3), (63, 1024, 16, 1, 1), (31, 1023, 16, 31, 9), (17, 1020, 5, 17, 16), (300, 256, 8, 8, 4),
          (100, 340, 7, 17, 2), (33, 1016, 8, 2, 1), (150, 60, 16, 5, 2)]


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,G,g", SHAPES)
def test_picks_and_weights(T, E, k, G, g, dtype, sigmoid, with_bias):
    logits = draw(T, E, T + E, dtype)
    bias = steps(E, T) if with_bias else None
    for group_max in (False, True):
        check(logits, k, n_group=G, topk_group=g, bias=bias, sigmoid=sigmoid, group_max=group_max, renormalise=group_max ^ (E % 2 == 0), scale=2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_ties_and_neighbours(sigmoid):
    """Equal logits, equal biases, scores that fp32 does not tell apart, scores that saturate."""
    g = torch.Generator(device=DEV).manual_seed(3)
    E = 64
    few = torch.randint(0, 4, (200, E), generator=g, device=DEV).float() * 0.5
    check(few, 8, n_group=8, topk_group=3, sigmoid=sigmoid)
    check(few, 8, n_group=8, topk_group=3, sigmoid=sigmoid, bias=torch.zeros(E, device=DEV))
    check(few, 8, n_group=8, topk_group=3, sigmoid=sigmoid, bias=steps(E, 1), group_max=True)
    check(torch.zeros(9, E, device=DEV), 8, n_group=4, topk_group=2, sigmoid=sigmoid, bias=torch.zeros(E, device=DEV))
    check(torch.zeros(9, E, device=DEV), 16, sigmoid=sigmoid, bias=torch.full((E,), 0.3, device=DEV))
    # a unit in the last place apart, in random order
    near = (1 + torch.randint(0, 6, (300, E), generator=g, device=DEV).float() * 2.0 ** -23)
    for bias in (None, torch.zeros(E, device=DEV), torch.full((E,), 3.0, device=DEV)):
        check(near, 8, n_group=8, topk_group=4, sigmoid=sigmoid, bias=bias)
    # a bias that makes up for the difference of two scores but for its own rounding
    l = draw(300, E, 8)
    for t in range(0, 300, 25):
        s = scores(l[t:t + 1].double(), sigmoid)[0]
        check(l[t:t + 1], 16, n_group=2, topk_group=2, sigmoid=sigmoid, bias=(s.max() + 0.25 - s).float())
    check(draw(100, E, 5, spread=30.0), 8, n_group=8, topk_group=4, sigmoid=sigmoid)
    check(draw(100, E, 6, spread=30.0), 8, n_group=8, topk_group=4, sigmoid=sigmoid, bias=steps(E, 2))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinities_nan_and_padding(dtype, sigmoid):
    E, k = 48, 6
    l = draw(40, E, 11, dtype)
    l[0] = float("-inf")
    l[1, 5:] = float("-inf")
    l[2] = torch.finfo(dtype).min
    l[3, ::3] = float("-inf")
    l[4] = -100.0
    bias = steps(E, 4)
    hard = bias.clone()
    hard[::2] = float("-inf")
    for kw in (dict(), dict(n_group=4, topk_group=2), dict(n_group=8, topk_group=2, group_max=True), dict(n_group=6, topk_group=3)):
        check(l, k, sigmoid=sigmoid, **kw)
        rows = slice(1, None) if not sigmoid else slice(0, None)  # softmax of a row of -inf: every score is NaN
        check(l[rows].contiguous(), k, sigmoid=sigmoid, bias=bias, **kw)
        check(l[rows].contiguous(), k, sigmoid=sigmoid, bias=hard, **kw)
    # NaN ranks last, in its own place
    l[6, 7] = float("nan")
    l[7] = float("nan")
    check(l, k, sigmoid=sigmoid)
    check(l, k, sigmoid=sigmoid, n_group=6, topk_group=3, group_max=True)
    # padding: whatever is there
    mask = torch.arange(40, device=DEV) % 3 != 0
    l[~mask] = float("nan")
    l[7] = 0.5
    l[6 + 1, 3] = 9.0
    r = check(l, k, sigmoid=sigmoid, mask=mask, n_group=6, topk_group=3)
    assert bool((r.ids[~mask] == -1).all()) and not bool(r.w[~mask].any())
    import expert_slot_cache_gb300 as M
    r8 = M.route_groups(l, k, 6, 3, token_mask=mask.to(torch.uint8), sigmoid=sigmoid)
    assert torch.equal(r.ids, r8.ids) and torch.equal(r.w, r8.w)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,G,g", [(8000, 512, 10, 8, 4), (500, 1024, 8, 16, 4), (300, 512, 16, 8, 4), (300, 256, 16, 8, 4),
                                       (300, 128, 16, 8, 2), (300, 64, 16, 1, 1), (300, 64, 8, 1, 1), (200, 72, 12, 2, 1),
                                       (200, 1024, 16, 32, 1), (200, 496, 16, 31, 1)])
def test_few_lanes_and_many_rounds(T, E, k, G, g, dtype, ties):
    """Picks out of few lanes' experts, about as many lanes as picks; more tokens than warps, some of them padding."""
    logits = draw(T, E, T + E + k, dtype)
    if ties:
        logits = torch.round(logits * 2) / 2
    mask = torch.rand(T, device=DEV, generator=torch.Generator(device=DEV).manual_seed(E)) > 0.1
    check(logits, k, n_group=G, topk_group=g, bias=steps(E, k), sigmoid=True, mask=mask, scale=2.5)
    check(logits, k, n_group=G, topk_group=g, group_max=True, renormalise=False, mask=mask)


def test_against_the_router():
    """Without groups, bias and scale: the picks and weights of the router that takes x."""
    import expert_slot_cache_gb300 as M
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(70, 256, generator=g, device=DEV).to(torch.bfloat16)
    wr = (torch.randn(256, 32, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    ids, w, logits = M.route(x, wr, 4, return_logits=True)
    r = M.route_groups(logits, 4)
    assert torch.equal(ids, r.ids) and torch.allclose(w, r.w, rtol=1e-5, atol=0)


def test_a_large_batch():
    l = draw(9000, 128, 21)
    check(l, 8, n_group=8, topk_group=4, bias=steps(128, 9), sigmoid=True, scale=2.5)


# --- the gradient -------------------------------------------------------------------------------------------------

def plain_grad(logits, ids, gw, sigmoid, renormalise, scale):
    """The formula (fp64) and the size of its terms."""
    l = logits.double().cpu()
    T, E = l.shape
    ids, gw = ids.cpu(), gw.double().cpu()
    grad, mag = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        on = (ids[t] >= 0) & (ids[t] < E)
        i, g = ids[t][on].long(), gw[t][on] * scale
        if not len(i):
            continue
        z = l[t][i]
        if renormalise:
            if bool(torch.isneginf(z).all()):
                continue
            q = torch.softmax(torch.nn.functional.logsigmoid(z) if sigmoid else z, 0)
            jac = torch.sigmoid(-z) if sigmoid else torch.ones_like(z)
            grad[t].index_add_(0, i, q * (g - (q * g).sum()) * jac)
            mag[t].index_add_(0, i, q * (g.abs() + (q * g.abs()).sum()) * jac)
        elif sigmoid:
            grad[t].index_add_(0, i, g * torch.sigmoid(z) * torch.sigmoid(-z))
            # a pick that is there twice: each term is rounded by itself, their sum may cancel
            mag[t].index_add_(0, i, g.abs() * torch.sigmoid(z) * torch.sigmoid(-z))
        else:
            s = torch.softmax(l[t], 0)
            G = torch.zeros(E, dtype=torch.float64).index_add_(0, i, g)
            A = torch.zeros(E, dtype=torch.float64).index_add_(0, i, g.abs())
            grad[t] = s * (G - (s * G).sum())
            mag[t] = s * (A + (s * A).sum())
    return grad, mag


def check_grad(logits, ids, gw, sigmoid, renormalise, scale=2.5):
    import expert_slot_cache_gb300 as M
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = M.route_groups_grad(logits, ids, gw, sigmoid, renormalise, scale, dev_status=st)
    grad, mag = plain_grad(logits, ids, gw, sigmoid, renormalise, scale)
    tol = 2e-5 * mag + 1e-37 + (2.0 ** -8 * grad.abs() if logits.dtype == torch.bfloat16 else 0)
    err = (got.double().cpu() - grad).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    again = M.route_groups_grad(logits, ids, gw, sigmoid, renormalise, scale)
    assert torch.equal(got, again)
    return got, int(st.item())


@pytest.mark.parametrize("sigmoid,renormalise", [(False, True), (False, False), (True, True), (True, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (7, 33, 2), (64, 512, 10), (255, 288, 8), (40, 1024, 16),
                                   (33, 1023, 9), (300, 130, 6), (5, 40, 16), (2500, 16, 2)])
def test_gradient(T, E, k, dtype, sigmoid, renormalise):
    logits = draw(T, E, T + E + 1, dtype)
    ids = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    g = torch.Generator(device=DEV).manual_seed(T)
    gw = torch.randn(T, k, generator=g, device=DEV)
    _, st = check_grad(logits, ids, gw, sigmoid, renormalise)
    assert st == 0
    # some picks left out, some tokens without any, some picks there twice (three times)
    ids[torch.rand(T, k, generator=g, device=DEV) < 0.2] = -1
    ids[::3] = -1
    if k >= 3:
        ids[1::4, 1] = ids[1::4, 0]
        ids[1::8, 2] = ids[1::8, 0]
    logits[::3] = float("nan")
    got, st = check_grad(logits, ids, gw, sigmoid, renormalise)
    assert st == 0 and not bool(got[::3].any())


def test_gradient_of_bad_picks():
    logits, ids = draw(6, 20, 1), torch.tensor([[0, 3], [20, 1], [-5, 2], [19, 18], [2, 2], [-1, 7]], dtype=torch.int32, device=DEV)
    gw = torch.ones(6, 2, device=DEV) * torch.tensor([1.0, -2.0], device=DEV)
    for sigmoid in (False, True):
        for renormalise in (False, True):
            _, st = check_grad(logits, ids, gw, sigmoid, renormalise)
            assert st == 1


def test_gradient_at_infinities():
    logits = draw(5, 24, 2)
    logits[0] = float("-inf")
    logits[1, 4:] = float("-inf")
    logits[3] = -200.0
    ids = torch.arange(6, dtype=torch.int32, device=DEV).repeat(5, 1)
    gw = draw(5, 6, 3)
    for sigmoid in (False, True):
        check_grad(logits, ids, gw, sigmoid, True)
    check_grad(logits, ids, gw, True, False)
    check_grad(logits[1:].contiguous(), ids[1:].contiguous(), gw[1:].contiguous(), False, False)


@pytest.mark.parametrize("sigmoid,renormalise", [(False, True), (False, False), (True, True), (True, False)])
def test_gradient_against_differences(sigmoid, renormalise):
    """Differences of the weights in 64 bits, the picks held: h^2 times a third derivative (< 1) and 1e-16 / h."""
    import expert_slot_cache_gb300 as M
    T, E, k, h = 4, 24, 5, 1e-5
    logits = draw(T, E, 31)
    ids, w = M.RouteGroups.apply(logits, k, 4, 2, None, None, sigmoid, False, renormalise, 1.5)
    gw = draw(T, k, 32)
    got = M.route_groups_grad(logits, ids, gw, sigmoid, renormalise, 1.5).double().cpu()
    l, i = logits.double().cpu(), ids.long().cpu()

    def loss(v):
        s = scores(v, sigmoid).gather(1, i)
        if renormalise:
            s = s / s.sum(1, keepdim=True)
        return (1.5 * s * gw.double().cpu()).sum(1)

    for e in range(E):
        d = torch.zeros_like(l)
        d[:, e] = h
        diff = (loss(l + d) - loss(l - d)) / (2 * h)
        assert bool(((got[:, e] - diff).abs() <= 1e-4 * diff.abs() + 1e-5).all())


def test_autograd():
    import expert_slot_cache_gb300 as M
    logits = draw(50, 64, 41).requires_grad_()
    mask = torch.arange(50, device=DEV) % 7 != 0
    ids, w = M.RouteGroups.apply(logits, 6, 8, 3, steps(64, 1), mask, True, False, True, 2.0)
    assert not ids.requires_grad and w.requires_grad
    gw = draw(50, 6, 42)
    (g,) = torch.autograd.grad((w * gw).sum(), logits, create_graph=True)
    want = M.route_groups_grad(logits.detach(), ids, gw, True, True, 2.0)
    assert torch.equal(g.detach(), want) and not bool(g[~mask].any())
    with pytest.raises(RuntimeError, match="second derivative"):
        (g * g).sum().backward()


def test_streams_graphs_and_unaligned_rows():
    import expert_slot_cache_gb300 as M
    buf = draw(1, 40 * 96 + 1, 51)[0]
    odd = buf[1:].view(40, 96)  # rows on 4 bytes
    check(odd, 8, n_group=4, topk_group=2, bias=steps(96, 3), sigmoid=True)
    ids = torch.topk(odd, 8, dim=1).indices.to(torch.int32)
    check_grad(odd, ids, draw(40, 8, 52), False, False)
    l, gw = draw(300, 128, 53), draw(300, 8, 54)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = M.route_groups(l, 8, 8, 4, sigmoid=True)
    wg = M.route_groups_grad(l, want.ids, gw, True)
    got = M.route_groups(l, 8, 8, 4, sigmoid=True, stream=s)
    gg = M.route_groups_grad(l, got.ids, gw, True, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(want.ids, got.ids) and torch.equal(want.w, got.w) and torch.equal(wg, gg)
    graph = torch.cuda.CUDAGraph()
    static = l.clone()
    with torch.cuda.graph(graph):
        r = M.route_groups(static, 8, 8, 4, sigmoid=True)
        rg = M.route_groups_grad(static, r.ids, gw, True)
    for seed in (60, 61):
        static.copy_(draw(300, 128, seed))
        graph.replay()
        w = M.route_groups(static, 8, 8, 4, sigmoid=True)
        assert torch.equal(r.ids, w.ids) and torch.equal(r.w, w.w)
        assert torch.equal(rg, M.route_groups_grad(static, w.ids, gw, True))
