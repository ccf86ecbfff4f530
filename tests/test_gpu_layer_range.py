"""The layer operators on inputs whose sizes differ widely: what small weights
and small inputs beside large ones add up to, against 64 bits.

Tolerances follow from what include/ep_layer.h says of each operator and the
rounding of fp32; test_gpu_layer.py has the units.
"""
import math

import pytest
import torch

from test_gpu_layer import F32, U, ep, gen, within  # noqa: F401  (ep: fixture)

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
