"""The experts' activation and its gradient over the whole range of a gate, infinities and NaN among them, against 64 bits.

A product of a row with one code or number that is not zero makes gate and up what the test wants, exactly. Tolerances: the
sigmoid of a gate is off by at most 8 * 2^-23 of itself, what it is multiplied with adds at most 4 roundings of 2^-24, and the
result is rounded to its type.
"""
import math

import pytest
import torch

from test_gpu_experts import E4M3, F32, TINY, U, ep, offsets_of, within  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan
LARGE = [INF, 3.38e38, 2.4e38, 2.3e38, 1e38, 1e20, 6.5e4, 1e3, 150.0, 104.5, 104.0, 103.0, 89.0, 88.0, 87.0, 50.0, 20.0, 17.0, 9.0, 1.0, 1e-3, 1e-30, 0.0]
GATES = LARGE + [-g for g in LARGE if not 88.5 < g < 1e3] + [NAN]
UPS = [1.0, -3.0, 1e-30, 1e30, 0.0]


def exact_act(gate, up):
    gate, up = gate.double(), up.double()
    return gate / (1 + torch.exp(-gate)) * up


def check_act(got, gate, up, dtype):
    want = exact_act(gate, up)
    most = torch.finfo(dtype).max * (1 + U[dtype] / 2)
    want = torch.where(want.abs() >= most, torch.sign(want) * INF, want)   # (what rounds past the largest number)
    within(got, want, ((8 + 2) * F32 + U[dtype]) * want.abs().nan_to_num(0, 0) + TINY[dtype])


def block_act(ep, gate, up, dtype, E):
    """act of the 16-bit block for gate and up [n] of the type, by E experts of 40 rows that are all the same."""
    F = -(-len(gate) // 8) * 8
    w = torch.zeros(E, 2 * F, 8, dtype=dtype, device="cuda")
    w[:, :len(gate), 0], w[:, F:F + len(gate), 0] = gate, up
    n = 40 * E
    x = torch.zeros(n, 8, dtype=dtype, device="cuda")
    x[:, 0] = 1
    act = torch.empty(n, F, dtype=dtype, device="cuda")
    ep.ep_expert_ffn(x, w, None, act, None, expert_offsets=offsets_of([40] * E))
    return act[:, :len(gate)]


def pairs(gates, ups, dtype):
    g, u = torch.meshgrid(torch.tensor(gates), torch.tensor(ups), indexing="ij")
    return g.reshape(-1).to(dtype).cuda(), u.reshape(-1).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E", [1, 30])
def test_block_at_large_gates(ep, dtype, E):
    gate, up = pairs(GATES, UPS, dtype)
    act = block_act(ep, gate, up, dtype, E)
    check_act(act, gate.expand_as(act), up.expand_as(act), dtype)


def fp8_act(ep, gate, up, dtype, E):
    """act of the fp8 product with the activation for gate and up [n] fp32 (rows), by E experts of the same n rows. The first
    block of inputs makes gates and the second ups; an infinite one is 448 times a scale that is not."""
    n, cols = len(gate), 640
    x = torch.zeros(E * n, 256, device="cuda")
    scales = torch.empty(n, 2, device="cuda")
    for k, v in enumerate((gate, up)):
        past = v.isinf()
        x.view(E, n, 256)[:, :, 128 * k] = torch.where(past, 448.0 * torch.sign(v), 1.0)
        scales[:, k] = torch.where(past, 3e38, v)
    w = torch.zeros(E, 2 * cols, 256, device="cuda")
    w[:, :cols, 0] = 1
    w[:, cols:, 128] = 1
    act = torch.empty(E * n, cols, dtype=dtype, device="cuda")
    ep.ep_expert_fp8(x.to(E4M3), scales.repeat(E, 1), w.to(E4M3), torch.ones(E, 2 * cols // 128, 2, device="cuda"), act,
                     expert_offsets=offsets_of([n] * E), activation=ep.EP_ACT_SWIGLU)
    return act.view(E, n, cols)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,most", [(1, 30), (48, 40), (48, 120)])   # tiles of 32 and 64 rows, and of rows as lanes
def test_fp8_at_large_gates(ep, dtype, E, most):
    gate, up = pairs(GATES, UPS, torch.float32)
    for at in range(0, len(gate), most):
        g, u = gate[at:at + most], up[at:at + most]
        if len(g) < most:
            g, u = gate[-most:], up[-most:]
        act = fp8_act(ep, g, u, dtype, E)
        # a NaN scale is that of both halves' sums: gate and up are NaN
        u = torch.where(g.isnan(), NAN, u)
        check_act(act, g[None, :, None].expand_as(act), u[None, :, None].expand_as(act), dtype)


def act_gradients(ep, gate, up, d, dtype, E):
    """(grad of gate, grad of up) [n, F] by E experts of 20 rows, for gate, up and gradients at act [F] of the type."""
    F = -(-len(gate) // 8) * 8
    n = 20 * E
    pad = torch.zeros(F - len(gate), dtype=dtype, device="cuda")
    gate_up = torch.cat((gate, pad, up, pad)).expand(n, 2 * F).contiguous()
    down = torch.zeros(E, 8, F, dtype=dtype, device="cuda")
    down[:, 0, :len(gate)] = d
    dy = torch.zeros(n, 8, dtype=dtype, device="cuda")
    dy[:, 0] = 1
    grads = torch.empty_like(gate_up)
    ep.ep_expert_ffn_backward(dy, None, gate_up, None, None, down, grads, expert_offsets=offsets_of([20] * E))
    return grads[:, :len(gate)], grads[:, F:F + len(gate)]


def check_gradients(got, gate, up, d, dtype, small=0.0):
    gate, up, d = gate.double(), up.double(), d.double()
    s = 1 / (1 + torch.exp(-gate))
    most = torch.finfo(dtype).max * (1 + U[dtype] / 2)
    slope = s * (1 + gate * (1 - s))
    # slope: its terms may cancel, and what s is off by counts gate times in 1 - s (from 17.4 on s is 1, exactly)
    terms = s * (1 + gate.abs() * (1 - s) + s * gate.abs().clamp(max=18)) * up.abs() * d.abs()
    for g, want, size in ((got[0], d * up * slope, terms), (got[1], d * (gate * s), (d * gate * s).abs())):
        want = torch.where(want.abs() >= most, torch.sign(want) * INF, want).expand_as(g)
        size = size.nan_to_num(0, 0).clamp(max=most)
        within(g, want, (16 * F32 * size).expand_as(g) + U[dtype] * want.abs().nan_to_num(0, 0) + TINY[dtype] + small)


def triples(gates, dtype):
    g, u, d = torch.meshgrid(torch.tensor(gates), torch.tensor([1.0, -7.0, 1e-4]), torch.tensor([1.0, 0.25, -1e-3]), indexing="ij")
    return [t.reshape(-1).to(dtype).cuda() for t in (g, u, d)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E", [1, 40])
def test_gradients_at_large_gates(ep, dtype, E):
    gate, up, d = triples(GATES, dtype)
    check_gradients(act_gradients(ep, gate, up, d, dtype, E), gate, up, d, dtype)


@pytest.mark.parametrize("E", [1, 40])
def test_gradients_of_large_products_stay_numbers(ep, E):
    """The gradient at act times up or gate may pass fp32's range where the sigmoid is small: their product is 0 or a number."""
    g, u, d = torch.meshgrid(torch.tensor([-3.38e38, -1e38, -1e4, -60.0, -5.0, 4.0, 1e4]), torch.tensor([1e30, -3e38, 2.0]),
                             torch.tensor([3.0, -1e9, 1e30, 3e38]), indexing="ij")
    gate, up, d = (t.reshape(-1).bfloat16().cuda() for t in (g, u, d))
    check_gradients(act_gradients(ep, gate, up, d, torch.bfloat16, E), gate, up, d, torch.bfloat16)


TAIL = [-88.5, -88.75, -89.0, -90.0, -92.5, -95.0, -99.0, -102.0, -103.5, -104.0, -105.0, -110.0, -150.0]


@pytest.mark.parametrize("E", [1, 30])
def test_block_at_far_negative_gates(ep, E):
    """Down to -110, where exp(-gate) is past fp32's range and the sigmoid below its normal numbers: large ups still show them."""
    gate, up = pairs(TAIL, [1.0, 1e10, -1e20, 1e30, 3e38], torch.bfloat16)
    act = block_act(ep, gate, up, torch.bfloat16, E)
    check_act(act, gate.expand_as(act), up.expand_as(act), torch.bfloat16)


@pytest.mark.parametrize("E,most", [(1, 30), (48, 40), (48, 65)])
def test_fp8_at_far_negative_gates(ep, E, most):
    gate, up = pairs(TAIL, [1.0, 1e10, -1e20, 1e30, 3e38], torch.float32)
    for g, u in ((gate[:most], up[:most]), (gate[-most:], up[-most:])):
        act = fp8_act(ep, g, u, torch.bfloat16, E)
        check_act(act, g[None, :, None].expand_as(act), u[None, :, None].expand_as(act), torch.bfloat16)


@pytest.mark.parametrize("E", [1, 40])
def test_gradients_at_far_negative_gates(ep, E):
    g, u, d = torch.meshgrid(torch.tensor(TAIL), torch.tensor([1.0, -1e20, 1e30]), torch.tensor([1.0, 1e-10, -1e20, 1e38]), indexing="ij")
    gate, up, d = (t.reshape(-1).bfloat16().cuda() for t in (g, u, d))
    # The sigmoid's factor 2^-124 is taken in two parts: slope * 2^124 * (up * 2^-62) may be a subnormal number, off by 2^-150, before
    # it is multiplied with d * 2^-62.
    check_gradients(act_gradients(ep, gate, up, d, torch.bfloat16, E), gate, up, d, torch.bfloat16, 2.0 ** -212 * d.double().abs())


def test_fp8_more_than_2_to_the_30_channels(ep):
    """Rows of x as lanes, and an output whose rows are longer than 2^31 bytes."""
    torch.cuda.empty_cache()
    n, O = 65, (1 << 30) + 512
    if torch.cuda.mem_get_info()[0] < 129 * O + n * 2 * O + (1 << 32):
        pytest.skip("needs 260 GiB")
    w = torch.zeros(1, O, 128, dtype=torch.uint8, device="cuda")
    some = torch.tensor([0, 5, 127, 128, 300, 511, 512, 1 << 29, O - 513, O - 1])
    codes = torch.randint(0, 0x70, (len(some), 128), generator=torch.Generator().manual_seed(1), dtype=torch.uint8)
    w[0, some.cuda()] = codes.cuda()
    x = torch.ones(n, 128, device="cuda").to(E4M3)
    scales = torch.arange(1, n + 1, device="cuda").float()[:, None]
    y = torch.full((n, O), NAN, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_fp8(x, scales, w.view(E4M3), torch.ones(1, O // 128, 1, device="cuda"), y)
    sums = codes.view(E4M3).double().sum(1)
    want = torch.arange(1, n + 1).double()[:, None] * sums
    # sums of 128 numbers of one sign, by a step of fp32 each at most, and two products
    within(y[:, some.cuda()], want, (130 * F32 + U[y.dtype]) * want)
    for part in (y[:, :4096], y[:, -4096:]):
        assert not part.isnan().any()
    del w, y
    torch.cuda.empty_cache()
