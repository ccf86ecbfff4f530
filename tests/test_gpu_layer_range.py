"""The layer operators on inputs whose sizes differ widely: what small weights
and small inputs beside large ones add up to, against 64 bits.

Tolerances follow from what include/ep_layer.h says of each operator and the
rounding of fp32; test_gpu_layer.py has the units.
"""
import math

import pytest
import torch

from test_gpu_layer import F32, U, attention_inputs, backward_reference, check_attention, ep, experts_inputs, gen, randn, within  # noqa: F401  (ep: fixture)

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
CACHES = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, E4M3), (torch.float16, E4M3)]


def weight_unit(cache):
    """(relative, absolute in units of the largest) error of an attention weight, as the header gives it."""
    return (2.0 ** -16, 0.0) if cache == torch.bfloat16 else (2.0 ** -22, 2.0 ** -36)


def attend(ep, q, kc, vc, table, lens, scale):
    out, lse = torch.full_like(q, math.nan), torch.empty(q.shape[:2], device="cuda")
    work = torch.empty(max(1, ep.ep_paged_attention_workspace(q, kc, table)), dtype=torch.uint8, device="cuda")
    ep.ep_paged_attention(q, kc, vc, table, lens, out, work, lse=lse, scale=scale)
    return out, lse


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("h,group", [(8, 1), (12, 3)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_values_that_cancel(ep, dtype, cache, h, group, d):
    """Values chosen so that each head's weighted sum is almost zero: the weights' rounding shows, the output's does not.
    Scores are exact (small integers), so nothing else is off. With shared heads the first of a group cancels."""
    g, N, n, scale = gen(d + h), 40, h // group, 0.25 * (64 / d) ** 0.5
    q = torch.randint(-2, 3, (1, h, d), generator=g).double()
    k = torch.randint(-4, 5, (N, n, d), generator=g).double() / 4
    s = torch.einsum("hd,khd->hk", q[0], k.repeat_interleave(group, 1)) * scale
    p = torch.softmax(s, 1)
    v = torch.randn(N, n, d, generator=g).to(cache).double()
    for j in range(n):
        big = p[j * group].topk(3).indices
        v[big, j] = 0.0
        for i in big:
            v[i, j] = (-(p[j * group] @ v[:, j]) / p[j * group, i]).to(cache).double()
    heads = v.repeat_interleave(group, 1)
    want, mag = torch.einsum("hk,khd->hd", p, heads), torch.einsum("hk,khd->hd", p, heads.abs())
    assert want[::group].abs().max() < 2.0 ** -9 * mag.max()
    kc, vc = (x.to(cache).view(1, N, n, d).cuda() for x in (k, v))
    out, _ = attend(ep, q.to(dtype).cuda(), kc, vc, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                    torch.tensor([N], dtype=torch.int32, device="cuda"), scale)
    relative, absolute = weight_unit(cache)
    # a score in units of log2, rounded three times and taken from the largest: off by 4 * 2^-24 of it; the power of two
    # itself and a score's product with the scale, 2^-21
    rel = relative + (s.abs().max() / math.log(2)) * 4 * 2.0 ** -24 + 2.0 ** -21 + N * F32
    within(out[0], want, mag * rel + absolute * heads.abs().sum(0) + want.abs() * U[dtype] * 1.01 + 2.0 ** -24)


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("above", [10, 18, 22])
def test_attention_sum_of_many_keys_beside_a_large_one(ep, dtype, cache, above):
    """One key `above` nats over 131071 others; its value is 0, so the output is the others' sum alone."""
    N, page, d, at = 131072, 64, 64, 70003
    kc, vc = torch.zeros(2, page, 1, d), torch.ones(2, page, 1, d)
    kc[1, at % page, 0, 0] = above
    vc[1, at % page] = 0.0
    table = torch.zeros(1, N // page, dtype=torch.int32)
    table[0, at // page] = 1
    q = torch.zeros(1, 1, d, dtype=dtype)
    q[0, 0, 0] = 1.0
    out, lse = attend(ep, q.cuda(), kc.to(cache).cuda(), vc.to(cache).cuda(), table.cuda(),
                      torch.tensor([N], dtype=torch.int32, device="cuda"), 1.0)
    others = (N - 1) * math.exp(-above)
    want = torch.full((d,), others / (1 + others), dtype=torch.float64)
    relative, absolute = weight_unit(cache)
    tol = want * (relative + above * 4 * F32 + 4096 * F32 + U[dtype] * 1.01) + absolute * N
    within(out[0, 0], want, tol)
    within(lse[0, 0], torch.tensor(above + math.log1p(others), dtype=torch.float64), 4096 * F32 + above * 4 * F32)


def experts_beside_large_inputs(counts, I, O, group, dtype, zeros, seed):
    """x, codes, scales, zero points, offsets and the exact y: one input of each group is 4096 with codes that equal the zero
    point, the others are odd multiples of a small step. All fp32 sums of these are exact (their 24 bits hold
    them), so y is the exact sum, rounded once."""
    bits, step = (8, 2.0 ** -6) if dtype == torch.bfloat16 else (10, 2.0 ** -7)
    g, rows, E, groups = gen(seed), sum(counts), len(counts), I // group
    x = (2 * torch.randint(0, 2 ** (bits - 1), (rows, I), generator=g) + 1).double() * step
    x *= torch.randint(0, 2, (rows, I), generator=g) * 2 - 1
    at = torch.arange(0, I, group) + torch.randint(0, group, (groups,), generator=g)
    x[:, at] = 4096.0
    assert torch.equal(x.to(dtype).double(), x)
    zero = torch.randint(0, 16, (E, groups, O), generator=g) if zeros else torch.full((E, groups, O), 8)
    code = torch.randint(0, 16, (E, O, I), generator=g)
    code[:, :, at] = zero.transpose(1, 2)
    scale = 2.0 ** torch.randint(-1, 2, (E, groups, O), generator=g).double()
    dense = (code - zero.transpose(1, 2).repeat_interleave(group, 2)) * scale.transpose(1, 2).repeat_interleave(group, 2)
    of = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    want = torch.stack([dense[of[r]] @ x[r] for r in range(rows)])
    off = torch.tensor([0] + list(counts)).cumsum(0).to(torch.int32)
    return (x.to(dtype).cuda(), (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8).cuda(), scale.to(dtype).cuda(),
            zero.to(torch.uint8).cuda() if zeros else None, off.cuda(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts", [[3, 2, 4, 1], [12], [20, 0, 17], [1], [7], [0, 2, 1, 5]])
@pytest.mark.parametrize("zeros", [False, True])
def test_experts_small_inputs_beside_large_ones(ep, dtype, group, counts, zeros):
    x, w, s, z, off, want = experts_beside_large_inputs(counts, 512, 160, group, dtype, zeros, group + sum(counts))
    y = torch.empty(want.shape, dtype=dtype, device="cuda")
    ep.ep_expert_w4(x, w, s, y, expert_offsets=off, zeros=z)
    assert torch.equal(y.cpu(), want.to(dtype))


def test_router_tokens_past_32_bits_of_threads(ep):
    """2^27 + 5 tokens, a warp each (groups of two experts): thread numbers pass 2^32."""
    T, K = (1 << 27) + 5, 2
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    rows = torch.randn(7, 4, generator=gen(70)).half().cuda()
    kw = dict(num_groups=2, topk_groups=1, renormalize=False)
    idx, w = torch.empty(7, K, dtype=torch.int64, device="cuda"), torch.empty(7, K, device="cuda")
    ep.ep_router_topk(rows, idx, w, **kw)
    at = torch.arange(T, device="cuda") % 7
    many_idx, many_w = torch.full((T, K), -7, dtype=torch.int64, device="cuda"), torch.full((T, K), math.nan, device="cuda")
    ep.ep_router_topk(rows[at], many_idx, many_w, **kw)
    for k in range(K):
        assert torch.equal(many_idx[:, k], idx[:, k][at]) and torch.equal(many_w[:, k], w[:, k][at])


def test_router_of_as_many_tokens_as_an_int_holds(ep):
    T = (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB")
    logits = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    idx, w = torch.full((T, 1), -7, dtype=torch.int64, device="cuda"), torch.zeros(T, 1, device="cuda")
    ep.ep_router_topk(logits, idx, w)
    assert int(idx.min()) == 0 and int(idx.max()) == 0
    assert float(w.min()) == 1.0 and float(w.max()) == 1.0


@pytest.mark.parametrize("dtype,cache,d", [(torch.bfloat16, torch.bfloat16, 8), (torch.float16, E4M3, 16), (torch.bfloat16, torch.bfloat16, 256)])
@pytest.mark.parametrize("short", [0, 1, 100])
def test_attention_window_at_the_end_of_2_to_the_31_places(ep, dtype, cache, d, short):
    """The longest table that is taken has 2^31 - 2 places (one page, named 1386 times): in the window's last chunk the places
    behind the end pass 2^31."""
    pages, page, g = 1386, 1549411, gen(d + short)
    assert pages * page == 2 ** 31 - 2
    kc, vc = (randn(g, 1, page, 1, d).to(cache) for _ in range(2))
    q = randn(g, 2, 4, d, dtype=dtype)
    table = torch.zeros(2, pages, dtype=torch.int32, device="cuda")
    lens = torch.tensor([2 ** 31 - 2 - short, 2 ** 31 - 1], dtype=torch.int64).to(torch.int32).cuda()
    check_attention(ep, q, kc, vc, table, lens, window=100)


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("above", [10, 18, 22])
def test_attention_sums_beside_a_large_key_in_each_of_many_sequences(ep, dtype, cache, above):
    """As above, with sequences enough that one block walks over each: what comes after the large key has it as its measure."""
    B, N, page, d, at = 400, 4096, 64, 64, 3
    kc, vc = torch.zeros(2, page, 1, d), torch.ones(2, page, 1, d)
    kc[1, at, 0, 0] = above
    vc[1, at] = 0.0
    table = torch.zeros(B, N // page, dtype=torch.int32)
    table[:, 0] = 1
    q = torch.zeros(B, 1, d, dtype=dtype)
    q[:, 0, 0] = 1.0
    out, _ = attend(ep, q.cuda(), kc.to(cache).cuda(), vc.to(cache).cuda(), table.cuda(),
                    torch.full((B,), N, dtype=torch.int32, device="cuda"), 1.0)
    others = (N - 1) * math.exp(-above)
    want = torch.full((B, d), others / (1 + others), dtype=torch.float64)
    relative, absolute = weight_unit(cache)
    within(out[:, 0], want, want * (relative + above * 4 * F32 + N * F32 + U[dtype] * 1.01) + absolute * N + 2.0 ** -25)


@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
def test_router_backward_of_experts_that_cannot_be_used(ep, score, renorm):
    """topk_idx may name experts that are masked (a routing made before the mask): they have no score and no gradient, in
    rows where nothing is left too."""
    E, K = 40, 4
    logits, grad_w = randn(gen(80), 5, E), randn(gen(81), 5, K)
    idx = torch.tensor([[0, 1, 2, 3], [39, 5, 5, 7], [4, 5, 6, 7], [8, 9, 10, 11], [-1, -1, -1, -1]])
    logits[0], logits[1], logits[4] = -math.inf, math.nan, -math.inf
    logits[2, 4:8] = -math.inf
    logits[3, 8], logits[3, 11] = -math.inf, math.nan
    grad = torch.full_like(logits, math.nan)
    ep.ep_router_topk_backward(logits, idx.cuda(), grad_w, grad, score=score, renormalize=renorm)
    want = torch.zeros(5, E, dtype=torch.float64)
    want[3] = backward_reference(logits[3:4], idx[3:4], grad_w[3:4], score, renorm, 1.0)[0]
    within(grad, want, 1e-5)


def test_attention_of_as_many_sequences_as_an_int_holds(ep):
    """2^31 - 1 sequences of one head, three of them with keys: the blocks' walk over the sequences ends, and finds them all."""
    B, page, d = (1 << 31) - 1, 1024, 8
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB")
    g = gen(90)
    kc, vc = (randn(g, 3, page, 1, d).bfloat16() for _ in range(2))
    some = torch.tensor([5, 1 << 30, B - 1])
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    q, out = torch.zeros(B, 1, d, dtype=torch.bfloat16, device="cuda"), torch.ones(B, 1, d, dtype=torch.bfloat16, device="cuda")
    few = dict(q=randn(g, 3, 1, d, dtype=torch.bfloat16), lens=torch.tensor([1000, 3, 700], dtype=torch.int32, device="cuda"),
               table=torch.tensor([[2], [0], [1]], dtype=torch.int32, device="cuda"))
    at = some.cuda()
    lens[at], table[at], q[at] = few["lens"], few["table"], few["q"]
    work = torch.empty(ep.ep_paged_attention_workspace(q, kc, table), dtype=torch.uint8, device="cuda")
    ep.ep_paged_attention(q, kc, vc, table, lens, out, work)
    want = check_attention(ep, few["q"], kc, vc, few["table"], few["lens"])
    assert bool(((out[at].float() - want.float()).abs() <= want.float().abs() * 2.0 ** -6 + 1e-6).all())
    out[at] = 0
    assert not bool(out.view(torch.int64).any())


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("scale", [2.0 ** 14, 2.0 ** 19, 2.0 ** 21, 2.0 ** 22, 2.0 ** 23, 2.0 ** 24])
def test_attention_scores_of_many_millions(ep, dtype, cache, scale):
    """Scores whose unit in the last place is above 1: one key takes all the weight, and nothing overflows on the way."""
    q, kc, vc, table, lens = attention_inputs(95, [300, 70, 1], 8, 2, 64, 16, dtype, cache)
    out = check_attention(ep, q, kc, vc, table, lens, scale=scale)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("rows", [3, 12])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("power", [-112, 120, 123])
def test_experts_near_the_ends_of_the_range(ep, rows, group, power):
    """bf16 inputs whose groups' sums pass fp32's range before the scale brings them back, and tiny ones: y is 2^power times what
    it is for inputs near 1."""
    x, w, s, z, off = experts_inputs(rows + group, [rows], 512, 48, group, torch.bfloat16, True)
    s = (s.float() * (2.0 ** -4 if power > 0 else 2.0 ** 4)).bfloat16()
    y, scaled = (torch.empty(rows, 48, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ep.ep_expert_w4(x, w, s, y, expert_offsets=off, zeros=z)
    ep.ep_expert_w4((x.double() * 2.0 ** power).bfloat16(), w, s, scaled, expert_offsets=off, zeros=z)
    assert bool(scaled.isfinite().all())
    assert torch.equal(scaled.double(), (y.double() * 2.0 ** power).bfloat16().double())
