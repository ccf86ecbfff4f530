"""The experts' products (ep_expert_fp8, ep_expert_ffn, ep_expert_ffn_backward of include/ep_layer.h) against their
definitions in 64 bits, at the sizes, layouts and types where they can go wrong.

Tolerances follow from the arithmetic: U is a type's unit of rounding (half a step, relative), a sum of n fp32 terms is
off by at most n * 2^-23 of the sum of magnitudes (every addition rounded or truncated), and what enters a function is
carried through its slope (that of silu is at most 1.1).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}   # half the smallest step
F32 = 2.0 ** -23
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
COUNTS = [[1], [0, 3, 0], [5, 0, 0, 17, 1], [16, 33], [130, 0, 64, 1], [300, 129], [0, 700, 2]]


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
    """Elementwise |got - want| <= tol (64-bit CPU tensors), infinities and NaN equal."""
    got, want = got.double().cpu(), want.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(want)
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i]} for {want[i]} +- {tol[i]}")


def offsets_of(counts):
    return torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()


def by_expert(counts, f):
    """Rows of f(e, slice) one expert after the other."""
    at, parts = 0, []
    for e, n in enumerate(counts):
        if n:
            parts.append(f(e, slice(at, at + n)))
        at += n
    return tuple(torch.cat(p) for p in zip(*parts))


def silu_parts(y, tol):
    """silu(gate) * up and its tolerance from gate and up [n, 2F] and theirs."""
    half = y.shape[1] // 2
    g, u, tg, tu = y[:, :half], y[:, half:], tol[:, :half], tol[:, half:]
    s = torch.nn.functional.silu(g)
    return s * u, 1.1 * tg * (u.abs() + tu) + s.abs() * tu + 8 * F32 * (s * u).abs()


# ------------------------------------------------------------------ fp8

def fp8_rows(g, n, I, dtype=E4M3, ue8m0=False, columns=False):
    x = torch.randn(n, I, generator=g)
    most = 448.0 if dtype == E4M3 else 57344.0
    s = x.view(n, -1, 128).abs().amax(2) / most
    if ue8m0:
        power = torch.ceil(torch.log2(s))
        codes, s = x / torch.exp2(power).repeat_interleave(128, 1), (power + 127).to(torch.uint8)
    else:
        codes = x / s.repeat_interleave(128, 1)
    codes = codes.clamp(-most, most).to(dtype).cuda()
    s = s.cuda()
    return codes, (s.t().contiguous().t() if columns else s)


def fp8_weights(g, E, O, I):
    w = (torch.randn(E, O, I, generator=g) * 100).clamp(-448, 448).to(E4M3).cuda()
    s = (torch.rand(E, -(-O // 128), I // 128, generator=g) + 0.5) / (100 * math.sqrt(I))
    return w, s.cuda()


def decoded(codes, scales):
    s = scales.double() if scales.dtype == torch.float32 else torch.exp2(scales.view(torch.uint8).double() - 127)
    return codes.double() * s.repeat_interleave(128, 1)


def fp8_reference(counts, x, xs, w, ws, swiglu):
    """(result, tolerance before the last rounding) in 64 bits."""
    rows, I = decoded(x, xs), x.shape[1]

    def one(e, at):
        wide = w[e].double() * ws[e].double().repeat_interleave(128, 0)[:w.shape[1]].repeat_interleave(128, 1)
        y = rows[at] @ wide.t()
        tol = (128 + 4 + I // 128) * F32 * (rows[at].abs() @ wide.abs().t())
        return silu_parts(y, tol) if swiglu else (y, tol)

    return by_expert(counts, one)


def run_fp8(ep, counts, I, O, swiglu=False, x_dtype=E4M3, ue8m0=False, columns=False, dtype=torch.bfloat16, seed=0):
    g = gen(seed + I + O + sum(counts))
    x, xs = fp8_rows(g, sum(counts), I, x_dtype, ue8m0, columns)
    w, ws = fp8_weights(g, len(counts), O, I)
    y = torch.full((sum(counts) + 1, O // 2 if swiglu else O), math.nan, dtype=dtype, device="cuda")
    ep.ep_expert_fp8(x, xs, w, ws, y[:-1], expert_offsets=offsets_of(counts),
                     activation=ep.EP_ACT_SWIGLU if swiglu else ep.EP_ACT_NONE)
    want, tol = fp8_reference(counts, x, xs, w, ws, swiglu)
    within(y[:-1], want, tol + U[dtype] * want.abs() + TINY[dtype])
    assert y[-1].isnan().all()   # (the row behind the last)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("I,O", [(128, 2), (128, 256), (640, 130), (1024, 520), (256, 70), (384, 384)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_fp8(ep, counts, I, O, swiglu):
    run_fp8(ep, counts, I, O, swiglu)


@pytest.mark.parametrize("x_dtype", [E4M3, E5M2])
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_fp8_types_and_scales(ep, x_dtype, ue8m0, columns, dtype):
    run_fp8(ep, [7, 0, 90], 768, 200, False, x_dtype, ue8m0, columns, dtype)


@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [16, 33], [300, 0, 129]])
@pytest.mark.parametrize("I,cols", [(128, 128), (640, 384), (256, 640)])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_fp8_quantised(ep, counts, I, cols, swiglu, mode):
    n, O = sum(counts), cols * (2 if swiglu else 1)
    g = gen(I + O + n)
    x, xs = fp8_rows(g, n, I)
    w, ws = fp8_weights(g, len(counts), O, I)
    y = torch.zeros(n, cols, dtype=E4M3, device="cuda")
    ys = torch.zeros(cols // 128, n, dtype=torch.uint8 if mode == 2 else torch.float32, device="cuda").t()
    ep.ep_expert_fp8(x, xs, w, ws, y, expert_offsets=offsets_of(counts), y_scales=ys, scale_mode=mode,
                     activation=ep.EP_ACT_SWIGLU if swiglu else ep.EP_ACT_NONE)
    want, tol = (t.cpu() for t in fp8_reference(counts, x, xs, w, ws, swiglu))
    s = torch.exp2(ys.double() - 127).cpu() if mode == 2 else ys.double().cpu()
    blocks, block_tol = want.abs().view(n, -1, 128).amax(2) / 448, tol.view(n, -1, 128).amax(2) / 448
    if mode == 0:
        within(s, blocks, block_tol + U[torch.float32] * blocks)
    else:   # the smallest power of two that is not below amax / 448, with what that may be off by
        assert torch.equal(torch.exp2(torch.round(torch.log2(s))), s)
        assert (s >= (blocks - block_tol) * (1 - F32)).all() and (s < 2 * (blocks + block_tol) * (1 + F32)).all()
    wide = s.repeat_interleave(128, 1)
    # a code is off by half a step: 2^-4 of it, or half of the smallest step, 2^-9
    within(y.double().cpu() * wide, want, tol + (want.abs() + tol) * 2.0 ** -4 + 2.0 ** -10 * wide)


def test_fp8_block_end_to_end(ep):
    """Both products, with what the first quantises: the second is held to the first's codes."""
    counts, H, F = [3, 0, 200, 40], 512, 384
    n, g = sum(counts), gen(5)
    x, xs = fp8_rows(g, n, H)
    up, ups = fp8_weights(g, 4, 2 * F, H)
    down, downs = fp8_weights(g, 4, H, F)
    act, scales = torch.empty(n, F, dtype=E4M3, device="cuda"), torch.empty(n, F // 128, device="cuda")
    y = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
    off = offsets_of(counts)
    ep.ep_expert_fp8(x, xs, up, ups, act, expert_offsets=off, y_scales=scales, activation=ep.EP_ACT_SWIGLU)
    ep.ep_expert_fp8(act, scales, down, downs, y, expert_offsets=off)
    want, tol = fp8_reference(counts, act, scales, down, downs, False)
    within(y, want, tol + U[torch.bfloat16] * want.abs())


# ------------------------------------------------------------------ gated block

def block_inputs(g, counts, H, F, dtype):
    E, n = len(counts), sum(counts)
    return (randn(g, n, H, dtype=dtype), randn(g, E, 2 * F, H, dtype=dtype, scale=H ** -0.5),
            randn(g, E, H, F, dtype=dtype, scale=F ** -0.5))


def product(counts, x, w):
    """(x W_e^T, sum of magnitudes) by expert."""
    return by_expert(counts, lambda e, at: (x[at].double() @ w[e].double().t(), x[at].double().abs() @ w[e].double().abs().t()))


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("H,F", [(8, 8), (64, 72), (200, 136), (512, 264)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_block(ep, counts, H, F, dtype):
    g, n = gen(sum(counts) + H), sum(counts)
    x, up, down = block_inputs(g, counts, H, F, dtype)
    act, y, gate_up = (torch.full((n + 1, w), math.nan, dtype=dtype, device="cuda") for w in (F, H, 2 * F))
    ep.ep_expert_ffn(x, up, down, act[:-1], y[:-1], gate_up=gate_up[:-1], expert_offsets=offsets_of(counts))
    want, size = product(counts, x, up)
    within(gate_up[:-1], want, H * F32 * size + U[dtype] * want.abs() + TINY[dtype])
    want, tol = silu_parts(want, H * F32 * size)
    within(act[:-1], want, tol + U[dtype] * want.abs() + TINY[dtype])
    want, size = product(counts, act[:-1], down)
    within(y[:-1], want, F * F32 * size + U[dtype] * want.abs() + TINY[dtype])
    for t in (act, y, gate_up):
        assert t[-1].isnan().all()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("H,F", [(8, 8), (64, 72), (200, 136), (512, 264)])
@pytest.mark.parametrize("dtype,grad_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                              (torch.bfloat16, torch.float32)])
def test_block_backward(ep, counts, H, F, dtype, grad_dtype):
    g, n, E = gen(sum(counts) + F), sum(counts), len(counts)
    x, up, down = block_inputs(g, counts, H, F, dtype)
    gate_up, act, dy = randn(g, n, 2 * F, dtype=dtype), randn(g, n, F, dtype=dtype), randn(g, n, H, dtype=dtype)
    d_gate_up, dx = (torch.full((n + 1, w), math.nan, dtype=dtype, device="cuda") for w in (2 * F, H))
    d_up, d_down = (torch.full_like(w, math.nan, dtype=grad_dtype) for w in (up, down))
    ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, d_gate_up[:-1], grad_x=dx[:-1], grad_w_gate_up=d_up,
                              grad_w_down=d_down, expert_offsets=offsets_of(counts))
    d_act, size = product(counts, dy, down.transpose(1, 2))
    tol = H * F32 * size
    gate, u = gate_up.double().chunk(2, 1)
    s = torch.sigmoid(gate)
    slopes = torch.cat((u * s * (1 + gate * (1 - s)), gate * s), 1)
    want, tol = slopes * d_act.repeat(1, 2), slopes.abs() * tol.repeat(1, 2)
    # s is off by 8 roundings; 1 + gate (1 - s) may cancel: its terms count
    terms = torch.cat((u.abs() * s * (1 + gate.abs() * (1 - s)), gate.abs() * s), 1) * d_act.abs().repeat(1, 2)
    within(d_gate_up[:-1], want, tol + 16 * F32 * terms + U[dtype] * want.abs() + TINY[dtype])
    assert d_gate_up[-1].isnan().all() and dx[-1].isnan().all()
    got = d_gate_up[:-1]
    want, size = product(counts, got, up.transpose(1, 2))
    within(dx[:-1], want, 2 * F * F32 * size + U[dtype] * want.abs() + TINY[dtype])
    at = 0
    for e, m in enumerate(counts):
        for grad, a, b in ((d_up[e], got[at:at + m], x[at:at + m]), (d_down[e], dy[at:at + m], act[at:at + m])):
            want, size = a.double().t() @ b.double(), a.double().abs().t() @ b.double().abs()
            within(grad, want, max(m, 1) * F32 * size + U[grad_dtype] * want.abs() + TINY[grad_dtype])
        at += m
