"""The layer operators (include/ep_layer.h) against plain implementations in
64 bits, at the sizes, masks, strides and types where they can go wrong.

Tolerances follow from the arithmetic: u(type) is the type's unit of rounding
(half a unit in the last place, relative), sums of n fp32 terms are off by at
most n * 2^-23 of the sum of magnitudes (every addition rounded or truncated),
and a factor that is rounded to 16 bits before a product adds that type's u.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -23


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_layout_gb300 as ep
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    ep.lib()
    return ep


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def within(got, want, tol):
    """Elementwise |got - want| <= tol (64-bit CPU tensors), infinities equal."""
    got, want = got.double().cpu(), want.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(want)
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i]} for {want[i]} +- {tol[i]}")


# ------------------------------------------------------------------ router

def router_reference(logits, K, score, renorm, scale, bias=None, groups=1, keep=1, group_top=1):
    """(idx, weights) by Python loops over rows, float64; keys that come from scores in float32 are compared
    in float64, so tests with such keys use logits whose scores are far apart."""
    l = logits.double().cpu().numpy()
    T, E = l.shape
    idx, w = np.full((T, K), -1, np.int64), np.zeros((T, K))
    by_score = bias is not None or (groups > 1 and group_top == 2)
    for t in range(T):
        row = np.where(np.isnan(l[t]), -np.inf, l[t])
        top = row.max()
        with np.errstate(all="ignore"):
            if score == 0:
                p = np.where(row == top, 1.0, np.exp(row - top)) if top > -np.inf else np.zeros(E)
                p = p / max(p.sum(), 1e-300)
            else:
                p = 1 / (1 + np.exp(-row))
        key = row.copy()
        if by_score:
            key = np.where(row > -np.inf, p + (0 if bias is None else bias.double().cpu().numpy()), -np.inf)
        if groups > 1:
            n = E // groups
            s = []
            for g in range(groups):
                part = np.sort(key[g * n:(g + 1) * n])[::-1]
                two = [v for v in part[:2] if v > -np.inf]
                s.append((sum(two) if two else -np.inf) if group_top == 2 else part[0])
            kept = sorted(range(groups), key=lambda g: (-s[g], g))[:keep]
            key = np.array([key[e] if e // n in kept else -np.inf for e in range(E)])
        chosen = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:K]
        for k, e in enumerate(chosen):
            idx[t, k] = e
        if chosen:
            if renorm and score == 0:
                v = np.where(row[chosen] == row[chosen].max(), 1.0, np.exp(row[chosen] - row[chosen].max()))
            elif renorm:   # ratios of sigmoids, the common factor out: exp of the logs' differences
                logs = -np.logaddexp(0, -row[chosen])
                v = np.exp(logs - logs.max())
            else:
                v = p[chosen]
            w[t, :len(chosen)] = scale * (v / v.sum() if renorm else v)
    return torch.from_numpy(idx), torch.from_numpy(w)


def router_tolerance(logits, w):
    """exp(l - m): the difference is off by up to 2^-24 |l - m|, exp itself by 2 units, and E terms add up."""
    l = logits.double().cpu()
    l = l[l.abs() < 1e30]
    spread = float(l.max() - l.min()) if l.numel() else 0.0
    return w.abs() * (2 * min(spread, 100.0) + 16 + 2 * math.sqrt(logits.shape[1])) * 2.0 ** -24 + 1e-38


def run_router(ep, logits, K, **kw):
    T = logits.shape[0]
    idx = torch.full((T, K), -7, dtype=torch.int64, device="cuda")
    w = torch.full((T, K), math.nan, device="cuda")
    ep.ep_router_topk(logits, idx, w, **kw)
    return idx.cpu(), w.cpu()


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 8), (5, 7, 3), (3, 33, 5), (130, 64, 6), (257, 256, 8),
                                   (9, 160, 32), (4, 1000, 8), (3, 4096, 32), (2, 3, 8), (6, 384, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
def test_router(ep, T, E, K, dtype, score, renorm):
    logits = randn(gen(T + E), T, E, dtype=dtype, scale=2.0)
    want_idx, want = router_reference(logits, K, score, renorm, 1.5)
    idx, w = run_router(ep, logits, K, score=score, renormalize=renorm, scale=1.5)
    assert torch.equal(idx, want_idx)
    within(w, want, router_tolerance(logits, want))


@pytest.mark.parametrize("groups,keep", [(2, 1), (4, 2), (8, 3), (8, 8), (32, 5)])
@pytest.mark.parametrize("score", [0, 1])
def test_router_groups(ep, groups, keep, score):
    logits = randn(gen(groups), 37, 256, dtype=torch.bfloat16, scale=2.0)
    want_idx, want = router_reference(logits, 6, score, True, 2.5, groups=groups, keep=keep)
    idx, w = run_router(ep, logits, 6, score=score, scale=2.5, num_groups=groups, topk_groups=keep)
    assert torch.equal(idx, want_idx)
    within(w, want, router_tolerance(logits, want))


@pytest.mark.parametrize("group_top", [1, 2])
def test_router_bias_and_group_sums(ep, group_top):
    # logits on a grid of 1/8 and biases on a grid of 1/512 set apart by expert: no two keys of a row closer than 1e-5
    g = gen(3)
    T, E = 64, 64
    logits = (torch.randint(-24, 25, (T, E), generator=g) / 8.0).cuda()
    bias = (torch.randperm(E, generator=g) / 512.0).cuda()
    key = torch.sigmoid(logits.double()) + bias.double()
    near = key.sort(1).values.diff(dim=1).min(1).values > 1e-5
    logits = logits[near]
    assert logits.shape[0] > 8
    want_idx, want = router_reference(logits, 4, 1, True, 1.0, bias, 8, 4, group_top)
    idx, w = run_router(ep, logits, 4, bias=bias, score=1, num_groups=8, topk_groups=4, group_top=group_top)
    if group_top == 2:   # sums of two keys may come closer: leave rows where the kept groups differ by rounding alone
        top2 = (torch.sigmoid(logits.double()) + bias.double()).view(-1, 8, 8).topk(2, dim=2).values.sum(2)
        far = (top2.sort(1).values.diff(dim=1).min(1).values > 1e-5).cpu()
        idx, w, want_idx, want = idx[far], w[far], want_idx[far], want[far]
        assert idx.shape[0] > 4
    assert torch.equal(idx, want_idx)
    within(w, want, router_tolerance(logits, want))


@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
def test_router_masked_infinite_and_lowest_rows(ep, score, renorm):
    inf, low = math.inf, torch.finfo(torch.float32).min
    rows = [[-inf] * 6, [-inf, 1, -inf, -inf, 2, -inf], [math.nan, 0.5, math.nan, 3, -inf, -2], [low] * 6,
            [low, 1, low, low, 0, low], [0.0, -0.0, 0.0, -0.0, 0.0, 0.0], [5, 5, 5, 5, 5, 5],
            [-300, -301, -302, -300, -310, -299], [80, 90, 100, 120, 85, 88]]
    if score == 0:
        rows.append([inf, 0, inf, 1, -inf, 3])
    logits = torch.tensor(rows, device="cuda")
    want_idx, want = router_reference(logits, 4, score, renorm, 1.0)
    idx, w = run_router(ep, logits, 4, score=score, renormalize=renorm)
    assert torch.equal(idx, want_idx)
    within(w, want, want.abs() * 400 * 2.0 ** -24 + 1e-38)


def test_router_strided_and_misaligned_rows(ep):
    wide = randn(gen(5), 40, 131, scale=2.0)
    for logits in (wide[:, 3:3 + 64], wide[::2, 1:1 + 100]):
        want_idx, want = router_reference(logits, 8, 0, True, 1.0)
        idx, w = run_router(ep, logits, 8)
        assert torch.equal(idx, want_idx)
        within(w, want, router_tolerance(logits, want))


@pytest.mark.parametrize("T,E,K", [(4096, 64, 8), (4099, 64, 6), (4097, 37, 8), (4098, 128, 16), (4101, 100, 9), (4096, 1, 1),
                                   (4103, 64, 9), (4102, 128, 17)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True)])
def test_router_many_tokens(ep, T, E, K, dtype, score, renorm):
    """Rows that share a warp (and ones whose K keeps them from it), some of them with few experts to use or none."""
    g = gen(T + E + K)
    logits = randn(g, T, E, dtype=dtype, scale=2.0)
    logits[torch.rand(T, E, generator=g).cuda() < 0.3] = -math.inf
    logits[1::7] = -math.inf
    want_idx, want = router_reference(logits, K, score, renorm, 1.5)
    idx, w = run_router(ep, logits, K, score=score, renormalize=renorm, scale=1.5)
    assert torch.equal(idx, want_idx)
    within(w, want, router_tolerance(logits, want))


@pytest.mark.parametrize("E,groups,keep", [(64, 8, 4), (64, 2, 1), (64, 32, 5), (128, 16, 3), (128, 8, 8), (96, 3, 2), (96, 12, 5)])
def test_router_many_tokens_in_groups(ep, E, groups, keep):
    T = 4099
    wide = randn(gen(E + groups), T, E + 3, dtype=torch.bfloat16, scale=2.0)
    for logits in (wide[:, :E].contiguous(), wide[:, 1:1 + E]):
        want_idx, want = router_reference(logits, 6, 1, True, 2.5, groups=groups, keep=keep, group_top=1)
        idx, w = run_router(ep, logits, 6, score=1, scale=2.5, num_groups=groups, topk_groups=keep, group_top=1)
        assert torch.equal(idx, want_idx)
        within(w, want, router_tolerance(logits, want))


@pytest.mark.parametrize("E,groups", [(64, 1), (64, 8), (128, 4)])
def test_router_many_tokens_with_a_bias(ep, E, groups):
    """As the bias test above: only rows with no two keys, and no two sums of a group's two largest, closer than 5e-6."""
    g = gen(17 + E + groups)
    logits = (torch.randint(-24, 25, (16384, E), generator=g) / 8.0).cuda()
    bias = (torch.randperm(E, generator=g) / 512.0).cuda()
    key = torch.sigmoid(logits.double()) + bias.double()
    near = key.sort(1).values.diff(dim=1).min(1).values > 5e-6
    if groups > 1:
        top2 = key.view(-1, groups, E // groups).topk(2, dim=2).values.sum(2)
        near &= top2.sort(1).values.diff(dim=1).min(1).values > 5e-6
    logits = logits[near]
    assert logits.shape[0] > 4096
    logits = logits[:4100]
    want_idx, want = router_reference(logits, 6, 1, True, 1.0, bias, groups, max(1, groups // 2), 2)
    idx, w = run_router(ep, logits, 6, bias=bias, score=1, num_groups=groups, topk_groups=max(1, groups // 2), group_top=2)
    assert torch.equal(idx, want_idx)
    within(w, want, router_tolerance(logits, want))


def test_router_feeds_the_layout(ep):
    """A router with unusable experts gives slots of -1, which the layout drops."""
    logits = randn(gen(6), 50, 16)
    logits[:, 3:] = -math.inf
    idx = torch.empty(50, 4, dtype=torch.int64, device="cuda")
    w = torch.empty(50, 4, device="cuda")
    ep.ep_router_topk(logits, idx, w)
    cnt, ntr = torch.empty(16, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    itr = torch.empty(50, 2, dtype=torch.uint8, device="cuda")
    off = torch.empty(17, dtype=torch.int32, device="cuda")
    h = ep.ep_layout(idx, 16, 2, cnt, ntr, itr, off)
    assert ep.ep_handle_query(h) == (150, 0)
    assert cnt.tolist() == [50, 50, 50] + [0] * 13
    h.destroy()


def backward_reference(logits, idx, g, score, renorm, scale):
    l = logits.double().cpu()
    l = torch.where(l.isnan(), -math.inf, l).requires_grad_()
    on = (idx >= 0) & (idx < l.shape[1])
    at = torch.where(on, idx, 0)
    p = torch.softmax(l, 1) if score == 0 else torch.sigmoid(l)
    w = torch.where(on, p.gather(1, at), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    (w * scale * g.double().cpu()).sum().backward()
    return l.grad


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 8, 8), (33, 256, 8), (7, 100, 5), (2, 4096, 32), (130, 64, 6)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
def test_router_backward(ep, T, E, K, dtype, score, renorm):
    gn = gen(T * E)
    logits = randn(gn, T, E, dtype=dtype, scale=2.0)
    idx = torch.stack([torch.randperm(E, generator=gn)[:K] for _ in range(T)])
    if T > 2 and K > 1:
        idx[0, 1] = -1
    g = randn(gn, T, K)
    grad = torch.full_like(logits, math.nan)
    ep.ep_router_topk_backward(logits, idx.cuda(), g, grad, score=score, renormalize=renorm, scale=1.5)
    want = backward_reference(logits, idx, g, score, renorm, 1.5)
    # each term is a product of scores and gradients of size <= |g|, with the error of a score (router_tolerance)
    top = 1.5 * g.abs().double().cpu().max()
    within(grad, want, want.abs() * U[dtype] * 1.01 + router_tolerance(logits, torch.ones(1)) * 4 * top
           + (2.0 ** -24 if dtype == torch.float16 else 0))


@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
def test_router_backward_differences(ep, score, renorm):
    """d(sum g w)/dl against central differences of the forward call itself (the chosen experts stay the same:
    their logits stand 4 above the rest). Error of a difference: h^2/6 of the third derivative, at most |g| in
    sum, plus the weights' 1e-6 over h."""
    gn = gen(11)
    T, E, K, h = 4, 24, 5, 2.0 ** -6
    logits = randn(gn, T, E)
    logits[:, :K] += 4 + 0.1 * torch.arange(K, device="cuda").flip(0)
    g = randn(gn, T, K)
    order = torch.full((T, E), 0.0, device="cuda")   # weight of each expert, whatever its place in the top K

    def loss(l):
        idx, w = (x.cuda() for x in run_router(ep, l, K, score=score, renormalize=renorm, scale=1.5))
        dense = torch.zeros_like(order).scatter_(1, idx, w)
        return (dense[:, :K].double() * g.double()).sum(1)

    idx0, _ = run_router(ep, logits, K, score=score, renormalize=renorm)
    assert all(set(r) == set(range(K)) for r in idx0.tolist())
    grad = torch.empty_like(logits)
    ep.ep_router_topk_backward(logits, torch.arange(K, device="cuda").expand(T, K).contiguous(), g, grad, score=score,
                               renormalize=renorm, scale=1.5)
    for e in range(E):
        step = torch.zeros_like(logits)
        step[:, e] = h
        diff = (loss(logits + step) - loss(logits - step)) / (2 * h)
        size = 1.5 * float(g.abs().sum(1).max())
        within(grad[:, e], diff, size * (h * h / 3 + 2e-6 / h))


def test_router_backward_repeated_and_invalid_experts(ep):
    logits = randn(gen(12), 3, 10)
    idx = torch.tensor([[2, 2, 2], [4, 10, -5], [-1, -1, -1]])
    g = randn(gen(13), 3, 3)
    for score, renorm in [(0, False), (0, True), (1, False), (1, True)]:
        grad = torch.full_like(logits, math.nan)
        ep.ep_router_topk_backward(logits, idx.cuda(), g, grad, score=score, renormalize=renorm)
        want = backward_reference(logits, idx, g, score, renorm, 1.0)
        want[2] = 0
        within(grad, want, 1e-5)


def test_router_backward_takes_a_slice_of_a_sort(ep):
    logits, g = randn(gen(16), 20, 64), randn(gen(17), 20, 6)
    order = logits.sort(dim=1, descending=True, stable=True).indices
    grad = torch.full_like(logits, math.nan)
    ep.ep_router_topk_backward(logits, order[:, :6], g, grad, renormalize=False)
    within(grad, backward_reference(logits, order[:, :6].cpu(), g, 0, False, 1.0), 1e-5)


@pytest.mark.parametrize("E,groups", [(60, 4), (96, 3), (1024, 8), (320, 10), (512, 16), (40, 5), (64, 2)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_router_group_sizes(ep, E, groups, group_top):
    """Groups that are and are not powers of two, rows in registers and in shared memory. A row's logits are all different,
    8 / E apart: no two scores are within rounding of each other."""
    g = gen(E)
    logits = torch.stack([(torch.randperm(E, generator=g) - E // 2) * (8.0 / E) for _ in range(23)]).cuda()
    logits[3, ::2] = -math.inf
    want_idx, want = router_reference(logits, 4, 1, True, 1.0, groups=groups, keep=2, group_top=group_top)
    idx, w = run_router(ep, logits, 4, score=1, num_groups=groups, topk_groups=2, group_top=group_top)
    if group_top == 2:   # the sums of two sigmoids of different groups may be that near
        top2 = torch.sigmoid(logits.double()).view(23, groups, -1).topk(2, dim=2).values.sum(2)
        far = (top2.sort(1).values.diff(dim=1).min(1).values > 1e-5).cpu()
        assert int(far.sum()) > 4
        idx, w, want_idx, want = idx[far], w[far], want_idx[far], want[far]
    assert torch.equal(idx, want_idx)
    within(w, want, router_tolerance(logits, want))


def test_router_backward_strided_rows(ep):
    wide = randn(gen(14), 12, 77)
    out = torch.full((12, 90), 5.0, device="cuda")
    logits, grad = wide[:, 5:69], out[:, 7:71]
    idx = torch.randint(0, 64, (12, 1), generator=gen(1)).repeat(1, 2)
    idx[:, 1] = (idx[:, 0] + 9) % 64
    g = randn(gen(15), 12, 2)
    ep.ep_router_topk_backward(logits, idx.cuda(), g, grad, renormalize=False)
    within(grad, backward_reference(logits, idx, g, 0, False, 1.0), 1e-5)
    assert bool((out[:, :7] == 5).all()) and bool((out[:, 71:] == 5).all())


# ------------------------------------------------------------------ append

def rotation_table(most, rot):
    half = rot // 2
    angle = torch.arange(most, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half) / max(half, 1))
    return torch.cat((angle.cos(), angle.sin()), 1).float().cuda()


def rotated(x, table, positions, rot, interleaved):
    """x [T, h, D] in float64, and the sum of the two products' magnitudes for the error bound."""
    x = x.double().cpu()
    t = table.double().cpu()[positions]
    half = rot // 2
    first = np.arange(half) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    cos, sin = t[:, None, :half], t[:, None, half:]
    out, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * cos - b * sin, b * cos + a * sin
    size[..., first], size[..., second] = (a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()
    return out, size


def cache_of(pages, page, n, d, dtype, heads_first, g):
    shape = (pages, n, page, d) if heads_first else (pages, page, n, d)
    c = randn(g, *shape).to(dtype)
    return c.transpose(1, 2) if heads_first else c


@pytest.mark.parametrize("T,h,n,d,rot,page,inter", [
    (1, 1, 1, 8, 8, 1, False), (1, 32, 8, 128, 128, 16, False), (37, 6, 2, 64, 64, 16, True),
    (19, 4, 4, 80, 40, 24, False), (23, 4, 1, 96, 48, 7, True), (64, 16, 2, 256, 128, 64, False),
    (5, 3, 3, 48, 20, 5, False), (5, 3, 3, 48, 20, 5, True), (9, 2, 1, 1024, 1024, 3, False), (7, 0, 2, 64, 64, 8, False),
    (11, 5, 2, 112, 0, 16, False), (6, 100, 3, 128, 126, 4, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads_first", [False, True])
def test_append(ep, T, h, n, d, rot, page, inter, dtype, fp8, heads_first):
    if fp8 and d % 16:
        pytest.skip("an e4m3 row is a multiple of 16 values")
    g = gen(T + d)
    qkv = randn(g, T, (h + 2 * n) * d + 8, dtype=dtype)[:, 8:]   # strided rows, as slices of one projection
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split((h * d, n * d, n * d), 1))
    pages, most = -(-T // page) + 3, 500
    positions = torch.randint(0, most, (T,), generator=g)
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 4:
        slots[3] = -1
    table = rotation_table(most, rot) if rot else None
    ct = torch.float8_e4m3fn if fp8 else dtype
    ks, vs = (0.02, 0.03) if fp8 else (1.0, 1.0)
    kc, vc = (cache_of(pages, page, n, d, ct, heads_first, g) for _ in range(2))
    before = [c.float().cpu() for c in (kc, vc)]
    q_out = torch.full((T, h, d), math.nan, dtype=dtype, device="cuda")
    err = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    ep.ep_kv_append(q if h else None, k, v, positions.cuda(), slots.cuda(), table, q_out if h else None, kc, vc,
                    interleaved=inter, k_scale=ks, v_scale=vs, device_error=err)
    assert err.item() == 0
    blank = torch.zeros(most, 0, device="cuda")
    want_k, size_k = rotated(k, table if rot else blank, positions, rot, inter)
    if h:
        want_q, size_q = rotated(q, table if rot else blank, positions, rot, inter)
        within(q_out, want_q, want_q.abs() * U[dtype] * 1.01 + size_q * 2 * F32 + 2.0 ** -25)
    touched = torch.zeros(pages, page, dtype=torch.bool)
    for c, old, x, size, scale in ((kc, before[0], want_k, size_k, ks),
                                   (vc, before[1], v.double().cpu(), torch.zeros(T, n, d), vs)):
        got = c.float().cpu().double()
        want = old.double()
        tol = torch.zeros_like(want)
        for t in range(T):
            if slots[t] < 0:
                continue
            at = (int(slots[t]) // page, int(slots[t]) % page)
            touched[at] = True
            y = x[t] / scale
            if fp8:   # half a unit of e4m3 (2^-4 relative, 2^-10 among its subnormals), saturating
                want[at] = y.clamp(-448, 448)
                tol[at] = (y.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 1e-5) + size[t] / scale * 4 * F32
            else:
                want[at] = y
                tol[at] = y.abs() * U[dtype] * 1.01 + size[t] * 2 * F32 + (2.0 ** -25 if rot else 0)
        within(got, want, tol)
        if not fp8 and rot == 0:
            assert torch.equal(got[touched], want[touched])


def test_append_values_are_copied_and_e4m3_codes_are_those_of_the_cast(ep):
    g = gen(40)
    T, n, d = 33, 2, 64
    k, v = randn(g, T, n, d, dtype=torch.bfloat16), randn(g, T, n, d, dtype=torch.bfloat16, scale=300.0)
    v[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1e30])
    slots = torch.randperm(48, generator=g)[:T].cuda()
    kc, vc = (torch.zeros(3, 16, n, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ep.ep_kv_append(None, k, v, slots, slots, None, None, kc, vc, k_scale=0.25, v_scale=2.0)
    for x, c, s in ((k, kc, 0.25), (v, vc, 2.0)):
        y = x.float() / s
        y = torch.where(y.isnan(), y, y.clamp(-448, 448)).to(torch.float8_e4m3fn)
        got = c.view(48, n, d)[slots.cpu()].float()
        want = y.float()
        assert torch.equal(got.nan_to_num(nan=999.0).cpu(), want.nan_to_num(nan=999.0).cpu())


def test_append_in_place_queries(ep):
    for d, rot, inter in ((128, 128, False), (80, 40, False), (48, 20, False), (64, 64, True)):
        g = gen(d)
        q = randn(g, 12, 7, d, dtype=torch.bfloat16)
        k, v = (randn(g, 12, 1, d, dtype=torch.bfloat16) for _ in range(2))
        kc, vc = (torch.zeros(2, 8, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        at = torch.arange(12, device="cuda")
        table = rotation_table(12, rot)
        apart = torch.empty_like(q)
        ep.ep_kv_append(q, k, v, at, at, table, apart, kc, vc, interleaved=inter)
        ep.ep_kv_append(q, k, v, at, at, table, q, kc, vc, interleaved=inter)
        assert torch.equal(q, apart)


def test_append_reports_bad_slots_and_positions(ep):
    g = gen(41)
    k, v = (randn(g, 6, 1, 64, dtype=torch.bfloat16) for _ in range(2))
    q = randn(g, 6, 2, 64, dtype=torch.bfloat16)
    table = rotation_table(10, 64)
    for slots, positions, bad in (([0, 1, 2, 3, 4, 16], [0] * 6, [5]), ([0, 1, -2, 3, 4, 5], [0] * 6, [2]),
                                  ([0, 1, 2, 3, 4, 5], [0, 10, 2, -1, 4, 5], [1, 3]),
                                  ([0, 1, 2, 3, 4, 1 << 40], [1 << 40, 1, 2, 3, 4, 5], [0, 5])):
        kc, vc = (torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q_out = torch.full_like(q, math.nan)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ep.ep_kv_append(q, k, v, torch.tensor(positions).cuda(), torch.tensor(slots).cuda(), table, q_out, kc, vc,
                        device_error=err)
        assert err.item() == ep.EP_ERR_INVALID_ARG
        assert bool(q_out.isfinite().all())
        for t in range(6):
            if not 0 <= positions[t] < 10:
                assert bool((q_out[t] == 0).all())
        flat = vc.view(16, 64).float().cpu()
        want = torch.zeros(16, 64)
        for t in range(6):
            if t not in bad:
                want[slots[t]] = v[t, 0].float().cpu()
        assert torch.equal(flat, want)


def test_append_past_32_bit_offsets(ep):
    """Slots whose element offset passes 2^31 and 2^32 (a cache of 5 * 2^30 e4m3 values)."""
    pages, page, n, d = 5 << 16, 16, 8, 128
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    kc, vc = (torch.zeros(pages, page, n, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
              for _ in range(2))
    k, v = (randn(gen(42), 4, n, d, dtype=torch.bfloat16) for _ in range(2))
    slots = torch.tensor([0, (1 << 31) // 1024 + 5, (1 << 32) // 1024 + 7, pages * page - 1], device="cuda")
    ep.ep_kv_append(None, k, v, slots, slots, None, None, kc, vc)
    for x, c in ((k, kc), (v, vc)):
        got = c.view(torch.uint8).view(-1, n, d)[slots].view(torch.float8_e4m3fn).float()
        assert torch.equal(got, x.float().to(torch.float8_e4m3fn).float())


# --------------------------------------------------------------- attention

def attention_reference(q, kc, vc, table, lens, scale, window=0, ks=1.0, vs=1.0, pages=None):
    """(out, lse, bound on the score error, sum p |v|) in float64 on the CPU."""
    B, h, d = q.shape
    P, page, n, _ = kc.shape
    q = q.double().cpu()
    out, lse = torch.zeros(B, h, d, dtype=torch.float64), torch.full((B, h), -math.inf, dtype=torch.float64)
    es, size = torch.zeros(B, h, dtype=torch.float64), torch.zeros(B, h, d, dtype=torch.float64)
    for b in range(B):
        length = min(max(int(lens[b]), 0), table.shape[1] * page)
        at = torch.arange(max(0, length - window) if window else 0, length)
        ids = table[b].long().cpu()[at // page]
        at, ids = at[(ids >= 0) & (ids < P)], ids[(ids >= 0) & (ids < P)]
        if not len(at):
            continue
        where = (ids.to(kc.device), (at % page).to(kc.device))
        if kc.dtype == torch.float8_e4m3fn:
            k, v = (c.view(torch.uint8)[where].view(torch.float8_e4m3fn).double().cpu() for c in (kc, vc))
        else:
            k, v = (c[where].double().cpu() for c in (kc, vc))
        for hh in range(h):
            kv = hh // (h // n)
            s = (k[:, kv] @ q[b, hh]) * scale * ks
            m = s.max()
            p = torch.exp(s - m)
            out[b, hh] = (p @ v[:, kv]) / p.sum() * vs
            size[b, hh] = (p @ v[:, kv].abs()) / p.sum() * vs
            lse[b, hh] = m + p.sum().log()
            es[b, hh] = ((k[:, kv].abs() @ q[b, hh].abs()).max() * abs(scale) * ks) * (d + 4) * F32 + s.abs().max() * F32
    return out, lse, es, size


def check_attention(ep, q, kc, vc, table, lens, window=0, ks=1.0, vs=1.0, scale=None):
    B, h, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out = torch.full_like(q, math.nan)
    lse = torch.full((B, h), math.nan, device="cuda")
    size = ep.ep_paged_attention_workspace(q, kc, table)
    work = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda")   # contents must not matter
    kw = dict(scale=scale, window=window, k_scale=ks, v_scale=vs)
    ep.ep_paged_attention(q, kc, vc, table, lens, out, work, lse=lse, **kw)
    want, want_lse, es, mag = attention_reference(q, kc, vc, table, lens, scale, window, ks, vs)
    keys = max(int(lens.max()), 1) if lens.numel() else 1
    # a weight is off by its score's error (twice: its own and the sum's), by its rounding to 16 bits, and by
    # the sums of `keys` terms
    rel = 2 * es[..., None] + 2 * U[q.dtype] + min(keys, 4096) * F32 + 1e-6
    within(out, want, mag * rel + want.abs() * U[q.dtype] * 1.01 + 2.0 ** -24)
    within(lse, want_lse, es + min(keys, 4096) * F32 + 2e-6 + torch.where(want_lse.isfinite(), want_lse.abs(), 0.0) * F32)
    again = torch.full_like(q, math.nan)
    ep.ep_paged_attention(q, kc, vc, table, lens, again, work, **kw)     # same bits, without lse too
    assert torch.equal(out, again)
    return out


def attention_inputs(seed, lens, h, n, d, page, dtype, cache=None, heads_first=False, width=None, qscale=1.5):
    g = gen(seed)
    B = len(lens)
    lens = torch.tensor(lens, dtype=torch.int32)
    width = width or max(1, -(-int(lens.max()) // page))
    pages = B * width + 2
    kc, vc = (cache_of(pages, page, n, d, cache or dtype, heads_first, g) for _ in range(2))
    table = torch.randperm(pages, generator=g)[:B * width].to(torch.int32).view(B, width)
    q = randn(g, B, h, d, dtype=dtype, scale=qscale)
    return q, kc, vc, table.cuda(), lens.cuda()


@pytest.mark.parametrize("h,n,d", [(1, 1, 64), (8, 8, 128), (32, 8, 128), (8, 1, 64), (7, 1, 80), (20, 4, 96),
                                   (16, 1, 128), (17, 1, 128), (40, 1, 64), (64, 1, 256), (6, 2, 256), (3, 3, 8),
                                   (4, 2, 200), (12, 4, 40), (128, 8, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_heads(ep, h, n, d, dtype):
    args = attention_inputs(h * d, [1, 0, 77, 300, 16], h, n, d, 16, dtype)
    check_attention(ep, *args)


@pytest.mark.parametrize("lens", [[1], [2], [15, 16, 17], [63, 64, 65], [0], [0, 0, 0], [127, 128, 129, 255, 256, 257],
                                  [1000], [1, 4097], [0, 513, 0, 1], [20000, 3], [-4, 5]])
@pytest.mark.parametrize("page", [1, 16, 24, 64, 256])
def test_attention_lengths_and_pages(ep, lens, page):
    args = attention_inputs(sum(lens) + page, lens, 8, 2, 64, page, torch.bfloat16)
    check_attention(ep, *args)


@pytest.mark.parametrize("d", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads_first", [False, True])
def test_attention_e4m3_cache(ep, d, dtype, heads_first):
    args = attention_inputs(d, [5, 200, 0, 64], 16, 2, d, 16, dtype, torch.float8_e4m3fn, heads_first)
    check_attention(ep, *args, ks=0.5, vs=1.5)


def test_attention_e4m3_cache_small_and_large_queries(ep):
    """Queries far outside fp16's range: bf16 q times e4m3 keys keeps q's relative precision."""
    for size in (2.0 ** 40, 2.0 ** -40, 2.0 ** -100):
        q, kc, vc, table, lens = attention_inputs(7, [100, 33], 8, 2, 64, 16, torch.bfloat16, torch.float8_e4m3fn)
        check_attention(ep, (q.float() * size).bfloat16(), kc, vc, table, lens, scale=0.125 / size)
    q = torch.zeros_like(q)
    check_attention(ep, q, kc, vc, table, lens)


@pytest.mark.parametrize("window", [1, 5, 64, 100, 5000])
@pytest.mark.parametrize("page", [16, 24])
def test_attention_window(ep, window, page):
    args = attention_inputs(window, [1, 64, 99, 100, 101, 1500, 0], 8, 2, 128, page, torch.bfloat16)
    q, kc, vc, table, lens = args
    for b in range(len(lens)):   # pages before the window are gone
        first = max(0, int(lens[b]) - window) // page
        table[b, :first] = -1
    check_attention(ep, q, kc, vc, table, lens, window=window)


def test_attention_masked_pages(ep):
    q, kc, vc, table, lens = attention_inputs(21, [100, 100, 100, 1], 8, 2, 64, 16, torch.bfloat16)
    table[0, 2] = -1
    table[1, 0], table[1, 6] = kc.shape[0], 2 ** 31 - 1      # past the cache
    table[2, :] = -7                                         # nothing left
    table[3, 0] = -1
    out = check_attention(ep, q, kc, vc, table, lens)
    assert bool((out[2:] == 0).all())


@pytest.mark.parametrize("cache", [None, torch.float8_e4m3fn])
@pytest.mark.parametrize("page", [16, 64])
def test_attention_ignores_what_lies_behind_the_end(ep, cache, page):
    """NaN and infinities in the slots behind each sequence's end and in unused pages."""
    lens = [1, 17, 63, 64, 100, 0]
    q, kc, vc, table, lens = attention_inputs(22, lens, 8, 2, 128, page, torch.bfloat16, cache)
    clean = check_attention(ep, q, kc, vc, table, lens)
    used = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b in range(len(lens)):
        for i in range(int(lens[b])):
            used[table[b, i // page].item(), i % page] = True
    bad = (~used).cuda()
    for c in (kc, vc):
        if cache is None:
            c[bad] = math.nan
            c[bad.nonzero()[0, 0], bad.nonzero()[0, 1], :, ::2] = math.inf
        else:
            c.view(torch.uint8)[bad] = 0x7F
    out = torch.empty_like(q)
    work = torch.empty(max(1, ep.ep_paged_attention_workspace(q, kc, table)), dtype=torch.uint8, device="cuda")
    ep.ep_paged_attention(q, kc, vc, table, lens, out, work)
    assert torch.equal(out, clean)


def test_attention_table_garbage_behind_the_end_and_wide_tables(ep):
    q, kc, vc, table, lens = attention_inputs(23, [40, 3, 0], 4, 4, 64, 16, torch.float16, width=60)
    for b in range(3):
        table[b, -(-int(lens[b]) // 16):] = 10 ** 9
    check_attention(ep, q, kc, vc, table, lens)
    lens[1] = 10 ** 9      # longer than its pages: taken as all of them, here with unusable ones masked
    check_attention(ep, q, kc, vc, table, lens)


def test_attention_strided_queries_and_outputs(ep):
    q, kc, vc, table, lens = attention_inputs(24, [70, 9], 8, 2, 64, 16, torch.bfloat16)
    wide = torch.zeros(2, 8 * 64 + 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:64 + 512] = q.flatten(1)
    strided = wide[:, 64:64 + 512].unflatten(1, (8, 64))
    big = torch.full((2, 8 * 64 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, 8:520].unflatten(1, (8, 64))
    work = torch.empty(max(1, ep.ep_paged_attention_workspace(q, kc, table)), dtype=torch.uint8, device="cuda")
    ep.ep_paged_attention(strided, kc, vc, torch.cat((table, table), 1)[:, :table.shape[1]], lens, out, work)
    assert torch.equal(out, check_attention(ep, q, kc, vc, table, lens))
    assert bool((big[:, :8] == 3).all()) and bool((big[:, 520:] == 3).all())


def test_attention_large_scores_and_peaks(ep):
    """Scores in the thousands: one key takes all the weight."""
    for qscale in (40.0, 400.0):
        args = attention_inputs(25, [300, 70], 8, 2, 64, 16, torch.bfloat16, qscale=qscale)
        check_attention(ep, *args)


def test_attention_many_short_sequences(ep):
    lens = [(7 * i) % 41 for i in range(700)]
    check_attention(ep, *attention_inputs(26, lens, 4, 2, 64, 16, torch.bfloat16))


@pytest.mark.parametrize("cache", [None, torch.float8_e4m3fn])
@pytest.mark.parametrize("h,n", [(4, 2), (9, 1), (8, 8)])
@pytest.mark.parametrize("seed", range(6))
def test_attention_very_uneven_lengths(ep, cache, h, n, seed):
    """Sequences of no keys, of one and of thousands side by side: shares that end anywhere in a unit, or before its first key."""
    rng = torch.Generator().manual_seed(100 + seed)
    lens = [int(torch.randint(0, top, (1,), generator=rng)) for top in (2, 70, 2, 5000, 300, 1, 130, 2, 2, 900, 40, 2000, 3)]
    lens = lens * (1 + seed % 3) + [1] * (seed * 7)
    check_attention(ep, *attention_inputs(200 + seed, lens, h, n, 64, 16, torch.bfloat16, cache))


def test_attention_long_sequence_splits(ep):
    for lens in ([100001], [70000, 1, 300]):
        check_attention(ep, *attention_inputs(27, lens, 8, 2, 64, 64, torch.float16))


def test_attention_past_32_bit_offsets(ep):
    """Pages whose element offset passes 2^32 in an e4m3 cache of 5 * 2^30 values."""
    pages, page, n, d = 5 << 16, 16, 8, 128
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    kc, vc = (torch.zeros(pages, page, n, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ids = [pages - 1, 3, (1 << 32) // (page * n * d) + 2, (1 << 31) // (page * n * d) + 1]
    for c in (kc, vc):
        for i in ids:
            c[i] = torch.randn(page, n, d, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    q = randn(gen(28), 1, 16, d, dtype=torch.bfloat16)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    check_attention(ep, q, kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), table,
                    torch.tensor([61], dtype=torch.int32, device="cuda"))


def test_attention_after_append(ep):
    """Tokens appended one by one are the keys that attention reads."""
    g = gen(29)
    n, h, d, page, steps = 2, 8, 64, 4, 11
    kc, vc = (torch.full((6, page, n, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[5, 1, 3]], dtype=torch.int32, device="cuda")
    cs = rotation_table(steps, d)
    ks, vs = [], []
    for t in range(steps):
        q, k, v = (randn(g, 1, x, d, dtype=torch.bfloat16) for x in (h, n, n))
        pos = torch.tensor([t], device="cuda")
        slot = table[0, t // page].long() * page + t % page
        q_out = torch.empty_like(q)
        ep.ep_kv_append(q, k, v, pos, slot.view(1), cs, q_out, kc, vc)
        lens = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        check_attention(ep, q_out, kc, vc, table, lens)


# ------------------------------------------------------------ 4-bit experts

def experts_inputs(seed, counts, I, O, group, dtype, zeros, xscale=1.0, pad=0):
    g = gen(seed)
    E, rows = len(counts), sum(counts)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts).cumsum(0)
    x = randn(g, rows + pad, I, dtype=dtype, scale=xscale)
    w = torch.randint(0, 256, (E, O, I // 2), dtype=torch.uint8, generator=g).cuda()
    s = ((torch.rand(E, I // group, O, generator=g) + 0.5) / (4.6 * math.sqrt(I))).to(dtype).cuda()
    z = torch.randint(0, 16, (E, I // group, O), dtype=torch.uint8, generator=g).cuda() if zeros else None
    return x, w, s, z, off.cuda()


def experts_reference(x, w, s, z, ranges, group, swiglu):
    """(y, bound without the final rounding) in float64; ranges: (expert, first row, end)."""
    rows, I = x.shape
    O = w.shape[1]
    cols = O // 2 if swiglu else O
    y, tol = torch.full((rows, cols), math.nan, dtype=torch.float64), torch.zeros(rows, cols, dtype=torch.float64)
    for e, a, b in ranges:
        if a >= b:
            continue
        code = torch.stack((w[e] & 15, w[e] >> 4), -1).view(O, I).double().cpu()
        zero = 8.0 if z is None else z[e].double().cpu().t().repeat_interleave(group, 1)
        dense = (code - zero) * s[e].double().cpu().t().repeat_interleave(group, 1)
        xs = x[a:b].double().cpu()
        v, err = xs @ dense.t(), (xs.abs() @ dense.abs().t()) * (I + 8) * F32
        if swiglu:
            gate, up, eg, eu = v[:, :cols], v[:, cols:], err[:, :cols], err[:, cols:]
            act = gate / (1 + torch.exp(-gate))
            v, err = act * up, 1.1 * eg * (up.abs() + eu) + act.abs() * eu + (act * up).abs() * 8 * F32
        y[a:b], tol[a:b] = v, err
    return y, tol


def check_experts(ep, x, w, s, z, off, group, swiglu=False, counts=None, ranges=None, y=None, offsets=True):
    rows = x.shape[0]
    cols = w.shape[1] // 2 if swiglu else w.shape[1]
    y = torch.full((rows, cols), math.nan, dtype=x.dtype, device="cuda") if y is None else y
    ep.ep_expert_w4(x, w, s, y, expert_offsets=off if offsets else None, expert_counts=counts, zeros=z,
                    activation=ep.EP_ACT_SWIGLU if swiglu else ep.EP_ACT_NONE)
    o = off.tolist()
    ranges = ranges or [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]
    want, tol = experts_reference(x, w, s, z, ranges, group, swiglu)
    within(y, want, torch.where(want.isnan(), 0.0, tol + want.abs() * U[x.dtype] * 1.01 + 2.0 ** -25))
    return y


@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [1, 2, 3, 0, 4], [8, 9], [16, 17, 0, 7], [33], [64, 1, 65], [150]])
@pytest.mark.parametrize("I,O,group", [(32, 1, 32), (128, 64, 128), (256, 130, 64), (96, 33, 32), (640, 200, 128),
                                       (1024, 256, 32), (192, 514, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("zeros", [False, True])
def test_experts(ep, counts, I, O, group, dtype, zeros):
    x, w, s, z, off = experts_inputs(I + O, counts, I, O, group, dtype, zeros)
    check_experts(ep, x, w, s, z, off, group)
    if O % 2 == 0:
        check_experts(ep, x, w, s, z, off, group, swiglu=True)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("rows", [1, 3, 8, 20])
def test_experts_dense_and_long_rows(ep, rows, swiglu):
    """One matrix without offsets; long rows, where a split over them would show."""
    for I, O, group in ((7168, 512, 128), (4096, 66, 64), (8192, 16, 32)):
        x, w, s, z, off = experts_inputs(rows, [rows], I, O, group, torch.bfloat16, True)
        check_experts(ep, x, w, s, z, off, group, swiglu=swiglu, offsets=False)


@pytest.mark.parametrize("rows", [9, 16, 17, 31, 32, 33, 64, 65, 100])
@pytest.mark.parametrize("experts", [1, 3])
def test_experts_shared_items(ep, rows, experts):
    """Numbers of items at which clusters of 8, 4 and 2 blocks share each, and one at which none does."""
    for O, I in ((512, 2048), (1030, 1024), (4096, 512)):
        counts = [rows] if experts == 1 else [rows // 2, 0, rows - rows // 2]
        x, w, s, z, off = experts_inputs(rows + O, counts, I, O, 128, torch.float16, True)
        check_experts(ep, x, w, s, z, off, 128)


def test_experts_strided_rows(ep):
    x, w, s, z, off = experts_inputs(50, [3, 4], 128, 36, 64, torch.float16, False)
    wide = torch.zeros(7, 160, dtype=torch.float16, device="cuda")
    wide[:, 16:144] = x
    big = torch.full((7, 45), 2.0, dtype=torch.float16, device="cuda")
    check_experts(ep, wide[:, 16:144], w, s, z, off, 64, y=big[:, 5:41])
    assert bool((big[:, :5] == 2).all()) and bool((big[:, 41:] == 2).all())


def test_experts_rows_of_aligned_and_strided_layouts(ep):
    """Only real rows are computed; pad rows and rows behind the last expert stay as they are."""
    counts, cap = [3, 0, 16, 9], 16
    x, w, s, z, _ = experts_inputs(51, [cap] * 4, 256, 70, 64, torch.bfloat16, True, pad=5)
    x[3:16], x[16:32] = math.nan, math.inf           # rows nobody asked for
    off = torch.arange(5, dtype=torch.int32, device="cuda") * cap
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    y = check_experts(ep, x, w, s, z, off, 64, counts=cnt, ranges=[(e, e * cap, e * cap + counts[e]) for e in range(4)])
    assert bool(y[3:32].isnan().all()) and bool(y[57:].isnan().all())
    # a count past the expert's range (a strided layout that dropped slots) ends at the range
    cnt[0] = 40
    x[:32] = 1.0
    check_experts(ep, x, w, s, z, off, 64, counts=cnt, ranges=[(0, 0, 16), (2, 32, 48), (3, 48, 57)])


def test_experts_offsets_past_the_rows_are_cut(ep):
    x, w, s, z, off = experts_inputs(52, [4, 6], 128, 40, 128, torch.bfloat16, False)
    want, tol = experts_reference(x, w, s, z, [(0, 0, 4), (1, 4, 7)], 128, False)
    y = torch.full((10, 40), math.nan, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_w4(x[:7], w, s, y[:7], expert_offsets=off)
    within(y[:7], want[:7], tol[:7] + want[:7].abs() * U[torch.bfloat16] * 1.01)
    assert bool(y[7:].isnan().all())


def test_experts_infinite_and_nan_rows_stay_in_their_rows(ep):
    x, w, s, z, off = experts_inputs(53, [5, 4], 256, 48, 64, torch.bfloat16, False)
    clean = check_experts(ep, x, w, s, z, off, 64)
    x[2, 7], x[6, 200] = math.nan, math.inf
    y = torch.empty_like(clean)
    ep.ep_expert_w4(x, w, s, y, expert_offsets=off)
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[2].isnan().all()) and not bool(y[6].isfinite().any())


@pytest.mark.parametrize("counts", [[8], [1, 1, 1, 1, 1, 1, 1, 1], [0, 5, 0, 3], [0, 0, 2, 1, 0, 4], [0, 0, 0]])
@pytest.mark.parametrize("I,O,group", [(32, 17, 32), (128, 64, 128), (384, 130, 128), (320, 50, 64), (1056, 256, 32), (2048, 1000, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("zeros", [False, True])
def test_experts_few_rows(ep, counts, I, O, group, dtype, zeros):
    """Up to 8 rows in all go through a kernel of their own; inputs over many powers of two."""
    x, w, s, z, off = experts_inputs(I + O + 1, counts, I, O, group, dtype, zeros, pad=0 if sum(counts) else 3)
    x *= 2.0 ** (torch.arange(x.shape[0], device="cuda")[:, None] % 5 * 2 - 6)
    x *= 2.0 ** (torch.arange(I, device="cuda") // 128 % 3 * 3.0)
    check_experts(ep, x, w, s, z, off, group)
    if O % 2 == 0:
        check_experts(ep, x / 32, w, s, z, off, group, swiglu=True)


def test_experts_few_rows_of_an_aligned_layout(ep):
    """Gaps between the experts' rows."""
    x, w, s, z, _ = experts_inputs(55, [2, 2, 0, 4], 256, 70, 64, torch.bfloat16, True)
    off = torch.tensor([0, 2, 4, 4, 8], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([1, 2, 0, 3], dtype=torch.int32, device="cuda")
    x[1], x[7] = math.nan, math.inf
    y = check_experts(ep, x, w, s, z, off, 64, counts=cnt, ranges=[(0, 0, 1), (1, 2, 4), (3, 4, 7)])
    assert bool(y[1].isnan().all()) and bool(y[7].isnan().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_experts_few_rows_infinite_and_nan(ep, dtype):
    x, w, s, z, off = experts_inputs(56, [5, 3], 256, 48, 64, dtype, False)
    clean = check_experts(ep, x, w, s, z, off, 64)
    x[2, 7], x[6, 200], x[7, 3] = math.nan, math.inf, -math.inf
    y = torch.empty_like(clean)
    ep.ep_expert_w4(x, w, s, y, expert_offsets=off)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[[2, 6, 7]].isnan().all())


@pytest.mark.parametrize("rows", [3, 12])
@pytest.mark.parametrize("power", [-100, -60, 60, 100])
def test_experts_powers_of_two(ep, rows, power):
    """bf16 rows times a power of two give outputs times the same power, bit for bit: nothing on the way over- or underflows."""
    x, w, s, z, off = experts_inputs(60, [rows], 512, 48, 64, torch.bfloat16, True)
    y, moved = (torch.empty(rows, 48, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ep.ep_expert_w4(x, w, s, y, expert_offsets=off, zeros=z)
    ep.ep_expert_w4(x * 2.0 ** power, w, s, moved, expert_offsets=off, zeros=z)
    assert torch.equal(moved, y * 2.0 ** power)


@pytest.mark.parametrize("swiglu", [False, True])
def test_experts_few_rows_of_many_outputs(ep, swiglu):
    """Tiles in several batches for each block, and more experts than threads."""
    x, w, s, z, off = experts_inputs(57, [2], 64, 90002, 64, torch.bfloat16, True)
    check_experts(ep, x, w, s, z, off, 64, swiglu=swiglu)
    x, w, s, z, off = experts_inputs(58, [0] * 600 + [2] + [0] * 30 + [1], 64, 20, 32, torch.float16, True)
    check_experts(ep, x, w, s, z, off, 32, swiglu=swiglu)


def test_experts_few_rows_past_32_bit_offsets(ep):
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    E, O, I = 160, 8192, 8192          # 5 GiB of codes
    w = torch.empty(E, O, I // 2, dtype=torch.uint8, device="cuda")
    w[150].random_(0, 256)
    s = torch.full((E, I // 128, O), 0.01, dtype=torch.bfloat16, device="cuda")
    x = randn(gen(59), 2, I, dtype=torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[151:] = 2
    y = torch.empty(2, O, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_w4(x, w, s, y, expert_offsets=off)
    part = slice(O - 300, O)
    want, tol = experts_reference(x, w[150:151, part], s[150:151, :, part], None, [(0, 0, 2)], 128, False)
    within(y[:, part], want, tol + want.abs() * U[torch.bfloat16] * 1.01)


def test_experts_weights_past_32_bit_offsets(ep):
    """Codes behind the first 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    E, O, I = 40, 32768, 8192          # 5 GiB of codes
    w = torch.empty(E, O, I // 2, dtype=torch.uint8, device="cuda")
    w[35].random_(0, 256)
    s = torch.full((E, I // 128, O), 0.01, dtype=torch.bfloat16, device="cuda")
    x = randn(gen(54), 3, I, dtype=torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[36:] = 3
    y = torch.empty(3, O, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_w4(x, w, s, y, expert_offsets=off)
    part = slice(O - 300, O)
    want, tol = experts_reference(x, w[35:36, part], s[35:36, :, part], None, [(0, 0, 3)], 128, False)
    within(y[:, part], want, tol + want.abs() * U[torch.bfloat16] * 1.01)


# ---------------------------------------------------------------- together

def test_refusals(ep):
    E = ep.EPError
    f = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    idx, w, logits = f(4, 2, dtype=torch.int64), f(4, 2, dtype=torch.float32), f(4, 8)
    for kw, err in ((dict(num_groups=3), E), (dict(num_groups=4, topk_groups=5), E), (dict(group_top=3), E),
                    (dict(score=7), E), (dict(scale=math.inf), E), (dict(bias=f(7, dtype=torch.float32)), ValueError)):
        with pytest.raises(err):
            ep.ep_router_topk(logits, idx, w, **kw)
    for bad in (lambda: ep.ep_router_topk(logits.double(), idx, w), lambda: ep.ep_router_topk(logits, idx.int(), w),
                lambda: ep.ep_router_topk(logits, idx[:3], w), lambda: ep.ep_router_topk(logits.t().contiguous().t(), idx, w),
                lambda: ep.ep_router_topk(logits.cpu(), idx, w),
                lambda: ep.ep_router_topk_backward(logits, idx, w, f(4, 8, dtype=torch.float32)),
                lambda: ep.ep_router_topk_backward(logits, idx, f(4, 2), logits)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(E):
        ep.ep_router_topk(logits, f(4, 33, dtype=torch.int64), f(4, 33, dtype=torch.float32))
    k, at, cs, c = f(4, 2, 64), f(4, dtype=torch.int64), f(9, 64, dtype=torch.float32), f(3, 8, 2, 64)
    append = lambda **kw: ep.ep_kv_append(**{**dict(q=f(4, 4, 64), k=k, v=k, positions=at, slots=at, cos_sin=cs,  # noqa: E731
                                                    q_out=f(4, 4, 64), k_cache=c, v_cache=c.clone()), **kw})
    for kw, err in ((dict(v=f(4, 3, 64)), ValueError), (dict(q_out=f(4, 4, 64, dtype=torch.float16)), ValueError),
                    (dict(positions=at.int()), ValueError), (dict(k_cache=f(3, 8, 4, 64)), ValueError),
                    (dict(cos_sin=f(9, 65, dtype=torch.float32)), E), (dict(cos_sin=f(9, 66, dtype=torch.float32)), E),
                    (dict(cos_sin=f(0, 64, dtype=torch.float32)), E), (dict(positions=None), E),
                    (dict(k_cache=c.half(), v_cache=c.half()), E), (dict(k=f(4, 2, 68)[..., :64], v=k), ValueError),
                    (dict(k_cache=c.to(torch.float8_e4m3fn), v_cache=c.to(torch.float8_e4m3fn), k_scale=0.0), E)):
        with pytest.raises(err):
            append(**kw)
    q, lens, table = f(4, 4, 64), f(4, dtype=torch.int32), f(4, 3, dtype=torch.int32)
    work = f(max(1, ep.ep_paged_attention_workspace(q, c, table)), dtype=torch.uint8)
    attend = lambda **kw: ep.ep_paged_attention(**{**dict(q=q, k_cache=c, v_cache=c, block_table=table, seq_lens=lens,  # noqa: E731
                                                          out=f(4, 4, 64), workspace=work), **kw})
    for kw, err in ((dict(q=f(4, 3, 64), out=f(4, 3, 64)), E), (dict(out=f(4, 4, 32)), ValueError),
                    (dict(seq_lens=lens.long()), ValueError), (dict(block_table=table.long()), ValueError),
                    (dict(block_table=table[:3]), ValueError), (dict(window=-1), E), (dict(scale=math.nan), E),
                    (dict(q=q.half(), out=q.half()), E), (dict(v_cache=f(3, 8, 2, 32)), ValueError),
                    (dict(lse=f(4, 4)), ValueError), (dict(q=q.cpu()), ValueError)):
        with pytest.raises(err):
            attend(**kw)
    with pytest.raises(ValueError):
        ep.ep_paged_attention_workspace(f(4, 3, 64), c, table)
    x, wt, sc, y = f(4, 128), f(2, 10, 64, dtype=torch.uint8), f(2, 1, 10), f(4, 10)
    off = f(3, dtype=torch.int32)
    expert = lambda **kw: ep.ep_expert_w4(**{**dict(x=x, weights=wt, scales=sc, y=y, expert_offsets=off), **kw})  # noqa: E731
    for kw, err in ((dict(expert_offsets=None), E), (dict(expert_offsets=off.long()), ValueError),
                    (dict(scales=f(2, 3, 10)), ValueError), (dict(scales=f(2, 8, 10)), E), (dict(activation=5), E),
                    (dict(activation=ep.EP_ACT_SWIGLU), ValueError), (dict(y=f(4, 9)), ValueError),
                    (dict(zeros=f(2, 1, 10)), ValueError), (dict(x=x.float()), ValueError),
                    (dict(weights=wt.view(torch.int8)), ValueError), (dict(expert_counts=off), ValueError)):
        with pytest.raises(err):
            expert(**kw)
    torch.cuda.synchronize()


def test_empty_calls(ep):
    f = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    ep.ep_router_topk(f(0, 8), f(0, 2, dtype=torch.int64), f(0, 2, dtype=torch.float32))
    ep.ep_router_topk_backward(f(0, 8), f(0, 2, dtype=torch.int64), f(0, 2, dtype=torch.float32), f(0, 8))
    c = f(3, 8, 2, 64)
    none = f(0, dtype=torch.int64)
    err = torch.full((1,), 3, dtype=torch.int32, device="cuda")
    ep.ep_kv_append(f(0, 4, 64), f(0, 2, 64), f(0, 2, 64), none, none, f(9, 64, dtype=torch.float32), f(0, 4, 64), c, c,
                    device_error=err)
    assert err.item() == 0
    q = f(0, 4, 64)
    ep.ep_paged_attention(q, c, c, f(0, 3, dtype=torch.int32), f(0, dtype=torch.int32), q, f(16, dtype=torch.uint8))
    q, out = f(2, 4, 64) + 1, f(2, 4, 64) + math.nan          # sequences without pages
    work = f(max(1, ep.ep_paged_attention_workspace(q, c, f(2, 0, dtype=torch.int32))), dtype=torch.uint8)
    ep.ep_paged_attention(q, f(0, 8, 2, 64), f(0, 8, 2, 64), f(2, 0, dtype=torch.int32), f(2, dtype=torch.int32) + 4, out,
                          work)
    assert bool((out == 0).all())
    ep.ep_expert_w4(f(0, 128), f(2, 10, 64, dtype=torch.uint8), f(2, 1, 10), f(0, 10), expert_offsets=f(3, dtype=torch.int32))


def test_on_another_stream_and_in_a_graph(ep):
    """All calls of a step captured once, replayed on new inputs."""
    g = gen(60)
    logits = randn(g, 9, 32)
    idx, wt = torch.empty(9, 4, dtype=torch.int64, device="cuda"), torch.empty(9, 4, device="cuda")
    q, kc, vc, table, lens = attention_inputs(61, [700, 33], 8, 2, 64, 16, torch.bfloat16)
    work = torch.empty(max(1, ep.ep_paged_attention_workspace(q, kc, table)), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    x, w, s, z, off = experts_inputs(62, [3, 0, 6], 256, 96, 64, torch.bfloat16, False)
    y = torch.empty(9, 96, dtype=torch.bfloat16, device="cuda")

    def step():
        ep.ep_router_topk(logits, idx, wt)
        ep.ep_paged_attention(q, kc, vc, table, lens, out, work)
        ep.ep_expert_w4(x, w, s, y, expert_offsets=off)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    first = [t.clone() for t in (idx, wt, out, y)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (idx, wt, out, y):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for t, want in zip((idx, wt, out, y), first):
        assert torch.equal(t, want)
    logits.copy_(randn(g, 9, 32))
    q.copy_(randn(g, *q.shape, dtype=torch.bfloat16))
    lens.copy_(torch.tensor([5, 64]))
    x.copy_(randn(g, *x.shape, dtype=torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (idx, wt, out, y)]
    step()
    torch.cuda.synchronize()
    for t, want in zip((idx, wt, out, y), replayed):
        assert torch.equal(t, want)


def dequantised(codes, scales, e, group):
    O, I = codes.shape[1], 2 * codes.shape[2]
    code = torch.stack((codes[e] & 15, codes[e] >> 4), -1).view(O, I).double().cpu()
    return (code - 8) * scales[e].double().cpu().t().repeat_interleave(group, 1)


def test_decode_layer_example(ep):
    """The example's layer, step by step, against each part's definition on the part's own inputs."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_layer
    T, group = 5, 64
    layer = decode_layer.DecodeLayer(T, hidden=256, heads=8, kv_heads=2, dim=64, experts=12, topk=3, inner=128, page=4,
                                     max_len=16, group=group)
    g = gen(70)
    for step in range(6):
        x = randn(g, T, 256, dtype=torch.bfloat16)
        cache = layer.k_cache.clone()
        y = layer.attention(x)
        h = decode_layer.norm(x)
        want, tol = experts_reference(h, layer.w_qkv, layer.s_qkv, None, [(0, 0, T)], group, False)
        within(layer.qkv, want, tol + want.abs() * U[torch.bfloat16] * 1.01)
        lens = layer.seq_lens
        assert lens.tolist() == [step + 1] * T
        changed = (layer.k_cache != cache).flatten(1).any(1).nonzero()[:, 0].tolist()
        assert sorted(changed) == sorted(layer.block_table[:, step // 4].tolist())
        check_attention(ep, layer.q, layer.k_cache, layer.v_cache, layer.block_table, lens)
        want, tol = experts_reference(layer.attended.flatten(1), layer.w_out, layer.s_out, None, [(0, 0, T)], group, False)
        within(layer.projected, want, tol + want.abs() * U[torch.bfloat16] * 1.01)
        assert torch.equal(y, x + layer.projected)

        z = layer.mixture(y)
        h = decode_layer.norm(y)
        want_idx, want_w = router_reference(h @ layer.gate.t(), 3, 0, True, 1.0)
        assert torch.equal(layer.idx.cpu(), want_idx)
        within(layer.weights, want_w, 1e-5)
        off = layer.offsets.tolist()
        assert off[-1] == 3 * T
        slots = sorted((int(e), t, k) for t in range(T) for k, e in enumerate(want_idx[t]))
        assert torch.equal(layer.received, torch.stack([h[t] for _, t, _ in slots]))
        ranges = [(e, off[e], off[e + 1]) for e in range(12)]
        want, tol = experts_reference(layer.received, layer.w_up, layer.s_up, None, ranges, group, True)
        within(layer.activated, want, tol + want.abs() * U[torch.bfloat16] * 1.01)
        want, tol = experts_reference(layer.activated, layer.w_down, layer.s_down, None, ranges, group, False)
        within(layer.returned, want, tol + want.abs() * U[torch.bfloat16] * 1.01)
        want = torch.zeros(T, 256, dtype=torch.float64)
        for row, (_, t, k) in enumerate(slots):
            want[t] += layer.weights[t, k].double().cpu() * layer.returned[row].double().cpu()
        within(layer.combined, want, want.abs() * U[torch.bfloat16] * 1.01 + 1e-6)
        assert torch.equal(z, y + layer.combined)
    layer.handle.destroy()


def test_decode_layer_example_runs_as_a_program():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decode_layer.py"), "--tokens", "8", "--steps", "4"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "outputs finite: True" in r.stdout


@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
def test_router_gradient_through_the_combine(ep, score, renorm):
    """Router, layout, dispatch, identity experts, combine, and all their gradients: the logits' gradient of
    sum(out * c) against autograd in 64 bits on the same rows."""
    g = gen(80)
    T, E, K, H = 40, 16, 4, 128
    x, c = randn(g, T, H, dtype=torch.bfloat16), randn(g, T, H, dtype=torch.bfloat16)
    logits = randn(g, T, E, scale=1.5)
    idx, w = torch.empty(T, K, dtype=torch.int64, device="cuda"), torch.empty(T, K, device="cuda")
    ep.ep_router_topk(logits, idx, w, score=score, renormalize=renorm, scale=1.25)
    cnt, ntr = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    itr, off = torch.empty(T, 1, dtype=torch.uint8, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    h = ep.ep_layout(idx, E, 1, cnt, ntr, itr, off)
    rows = torch.empty(T * K, H, dtype=torch.bfloat16, device="cuda")
    ep.ep_dispatch(h, x, ep.EP_DTYPE_BF16, rows, T * K)
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), cnt.long())
    y = (rows.float() * (1 + 0.1 * expert[:, None])).bfloat16()        # experts that differ
    grad_w = torch.empty(T, K, device="cuda")
    ep.ep_combine_backward(h, c, y, topk_weights=w, grad_topk_weights=grad_w)
    grad = torch.empty_like(logits)
    ep.ep_router_topk_backward(logits, idx, grad_w, grad, score=score, renormalize=renorm, scale=1.25)
    row_of = torch.empty(T, K, dtype=torch.int32, device="cuda")
    ep.ep_handle_copy_row_of_slot(h, row_of)
    dots = torch.einsum("tkh,th->tk", y[row_of.long()].double(), c.double()).cpu()
    want = backward_reference(logits, idx.cpu(), dots, score, renorm, 1.25)
    size = float(dots.abs().max())
    within(grad, want, size * 4e-5)     # the dots are fp32 sums of H products, the scores good to 1e-6
    h.destroy()
