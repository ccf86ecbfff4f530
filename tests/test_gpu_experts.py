"""The experts' products (ep_expert_fp8, ep_expert_ffn, ep_expert_ffn_backward of include/ep_layer.h) against their
definitions in 64 bits, at the sizes, layouts and types where they can go wrong.

Tolerances follow from the arithmetic: U is a type's unit of rounding (half a step, relative), a sum of n fp32 terms is
off by at most n * 2^-23 of the sum of magnitudes (every addition rounded or truncated), and what enters a function is
carried through its slope (that of silu is at most 1.1).
"""
import math
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


# ------------------------------------------------------------------ layouts, strides, sizes

def one_block(ep, counts, H, F, dtype=torch.bfloat16, offsets=None, expert_counts=None, rows=None, seed=0):
    """act and y of a block on rows [rows], others NaN before the call; (x, weights, act, y)."""
    g = gen(seed + H + F)
    n = rows if rows is not None else sum(counts)
    E = len(counts)
    x, up, down = randn(g, n, H, dtype=dtype), randn(g, E, 2 * F, H, dtype=dtype, scale=H ** -0.5), randn(g, E, H, F, dtype=dtype, scale=F ** -0.5)
    act, y = (torch.full((n, w), math.nan, dtype=dtype, device="cuda") for w in (F, H))
    ep.ep_expert_ffn(x, up, down, act, y, expert_offsets=offsets if offsets is not None else offsets_of(counts),
                     expert_counts=expert_counts)
    return x, up, down, act, y


def check_block_rows(x, up, down, act, y, owner):
    """Rows with an expert are its block's (through the act that is there), the others were not written."""
    dtype = x.dtype
    owner = torch.tensor(owner)
    for e in range(up.shape[0]):
        at = (owner == e).nonzero()[:, 0].cuda()
        if not len(at):
            continue
        g = x[at].double() @ up[e].double().t()
        want, tol = silu_parts(g, x.shape[1] * F32 * (x[at].double().abs() @ up[e].double().abs().t()))
        within(act[at], want, tol + U[dtype] * want.abs() + TINY[dtype])
        want, size = act[at].double() @ down[e].double().t(), act[at].double().abs() @ down[e].double().abs().t()
        within(y[at], want, act.shape[1] * F32 * size + U[dtype] * want.abs() + TINY[dtype])
    nobody = (owner < 0).nonzero()[:, 0].cuda()
    assert act[nobody].isnan().all() and y[nobody].isnan().all()


def owners(offsets, counts, rows):
    owner = [-1] * rows
    for e, n in enumerate(counts):
        for r in range(offsets[e], min(offsets[e] + n, rows)):
            owner[r] = e
    return owner


def test_rows_of_aligned_and_strided_layouts(ep):
    for offsets, counts in (([0, 128, 128, 256], [100, 0, 3]), ([0, 40, 80, 120], [40, 0, 17]), ([0, 300, 600, 900], [1, 300, 129])):
        off, cnt = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (offsets, counts))
        x, up, down, act, y = one_block(ep, counts, 136, 72, offsets=off, expert_counts=cnt, rows=offsets[-1])
        check_block_rows(x, up, down, act, y, owners(offsets, counts, offsets[-1]))


def test_offsets_past_the_rows_and_rows_of_nobody(ep):
    """Rows before the first and behind the last expert's belong to nobody; offsets past the rows are cut."""
    off = torch.tensor([5, 20, 20, 500], dtype=torch.int32, device="cuda")
    x, up, down, act, y = one_block(ep, [15, 0, 40], 64, 64, offsets=off, rows=60)
    check_block_rows(x, up, down, act, y, owners([5, 20, 20], [15, 0, 40], 60))


@pytest.mark.parametrize("E,rows", [(300, 700), (1024, 500), (1500, 3001), (4096, 900)])
def test_many_experts(ep, E, rows):
    g = gen(E)
    counts = torch.bincount(torch.randint(0, E, (rows,), generator=g), minlength=E).tolist()
    x, up, down, act, y = one_block(ep, counts, 32, 24)
    check_block_rows(x, up, down, act, y, [e for e, n in enumerate(counts) for _ in range(n)])
    n, I, O = rows, 128, 24
    x, xs = fp8_rows(g, n, I)
    w, ws = fp8_weights(g, E, O, I)
    y = torch.empty(n, O, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_fp8(x, xs, w, ws, y, expert_offsets=offsets_of(counts))
    want, tol = fp8_reference(counts, x, xs, w, ws, False)
    within(y, want, tol + U[y.dtype] * want.abs())
    gate_up, act, dy = (randn(g, n, k, dtype=torch.bfloat16) for k in (16, 8, 16))
    x, down = randn(g, n, 16, dtype=torch.bfloat16), randn(g, E, 16, 8, dtype=torch.bfloat16)
    dgu, dw = torch.empty_like(gate_up), torch.full((E, 16, 8), math.nan, device="cuda")
    ep.ep_expert_ffn_backward(dy, None, gate_up, act, None, down, dgu, grad_w_down=dw, expert_offsets=offsets_of(counts))
    at = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    pairs = dy.double()[:, :, None] * act.double()[:, None]
    want = torch.zeros(E, 16, 8, dtype=torch.float64, device="cuda").index_add_(0, at, pairs)
    size = torch.zeros_like(want).index_add_(0, at, pairs.abs())
    within(dw, want, max(counts) * F32 * size + U[torch.float32] * want.abs())


def strided(t, extra):
    """The same values with rows `extra` elements further apart."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), math.nan).to(t.dtype).cuda()
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def test_strided_rows(ep):
    counts, H, F = [70, 0, 9, 200], 72, 40
    g, n, off = gen(9), sum(counts), offsets_of(counts)
    x, up, down = block_inputs(g, counts, H, F, torch.bfloat16)
    gate_up, act, dy = (randn(g, n, k, dtype=torch.bfloat16) for k in (2 * F, F, H))

    def forward(f):
        outs = [f(torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")) for k in (F, H, 2 * F)]
        ep.ep_expert_ffn(f(x), up, down, outs[0], outs[1], gate_up=outs[2], expert_offsets=off)
        return outs

    def backward(f):
        outs = [f(torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")) for k in (2 * F, H)] + [torch.empty_like(up), torch.empty_like(down)]
        ep.ep_expert_ffn_backward(f(dy), f(x), f(gate_up), f(act), up, down, outs[0], outs[1], outs[2], outs[3], expert_offsets=off)
        return outs

    for call in (forward, backward):
        for a, b in zip(call(lambda t: t), call(lambda t: strided(t, 24))):
            assert torch.equal(a, b)
    x8, xs = fp8_rows(g, n, 256)
    w, ws = fp8_weights(g, 4, 200, 256)
    y, wide = torch.empty(n, 200, dtype=torch.bfloat16, device="cuda"), torch.full((n, 203), 7.0, dtype=torch.bfloat16, device="cuda")
    far = torch.zeros(n, 304, dtype=torch.uint8, device="cuda").view(E4M3)[:, :256]
    far.view(torch.uint8).copy_(x8.view(torch.uint8))
    scales = torch.zeros(n, 6, device="cuda")
    scales[:, 1::2][:, :2] = xs
    ep.ep_expert_fp8(x8, xs, w, ws, y, expert_offsets=off)
    ep.ep_expert_fp8(far, scales[:, 1:5:2], w, ws, wide[:, :200], expert_offsets=off)
    assert torch.equal(y, wide[:, :200]) and (wide[:, 200:] == 7).all()


@pytest.mark.parametrize("counts", [[3, 20, 9], [40, 150, 17], [300, 20, 100]])
def test_nan_and_infinity_stay_in_their_rows_and_experts(ep, counts):
    """A row of NaN, of another expert than most, and an expert whose weights are infinite touch nothing else."""
    H, F, n, g = 136, 72, sum(counts), gen(3)
    x, up, down = block_inputs(g, counts, H, F, torch.bfloat16)
    gate_up, act, dy = (randn(g, n, k, dtype=torch.bfloat16) for k in (2 * F, F, H))
    off = offsets_of(counts)

    def all_of(x, up, down, gate_up, act, dy):
        outs = [torch.empty(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H, 2 * F, 2 * F, H)] + [torch.empty_like(up), torch.empty_like(down)]
        ep.ep_expert_ffn(x, up, down, outs[0], outs[1], gate_up=outs[2], expert_offsets=off)
        ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, outs[3], outs[4], outs[5], outs[6], expert_offsets=off)
        return outs

    clean = all_of(x, up, down, gate_up, act, dy)
    bad = [t.clone() for t in (x, up, down, gate_up, act, dy)]
    first = counts[0]                       # the second expert: a row of NaN; the last expert: weights of infinity
    for t in (bad[0], bad[3], bad[4], bad[5]):
        t[first] = math.nan
    bad[1][2], bad[2][2] = math.inf, math.inf
    dirty = all_of(*bad)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[first] = False
    keep[first + counts[1]:] = False
    for a, b in zip(clean[:5], dirty[:5]):
        assert torch.equal(a[keep], b[keep])
        assert b[first].isnan().any()
    for a, b in zip(clean[5:], dirty[5:]):
        assert torch.equal(a[0], b[0]) and b[1].isnan().any()
    # fp8: a NaN code, a NaN scale
    x8, xs = fp8_rows(g, n, 256)
    w, ws = fp8_weights(g, 3, 256, 256)
    outs = []
    for k in range(3):
        c, s = x8.clone(), xs.clone()
        if k == 1:
            c.view(torch.uint8)[first, 130] = 0x7F
        if k == 2:
            s[first, 1] = math.nan
        y = torch.empty(n, 256, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_fp8(c, s, w, ws, y, expert_offsets=off)
        outs.append(y)
    keep = torch.arange(n, device="cuda") != first
    for y in outs[1:]:
        assert torch.equal(y[keep], outs[0][keep]) and y[first].isnan().all()


@pytest.mark.parametrize("counts", [[3], [1, 20], [100, 40], [300]])
def test_fp8_zero_blocks_and_extreme_scales(ep, counts):
    """Zero rows give zeros and scale 0; results near both ends of the output's range; scales far apart in one row."""
    g, n = gen(1), sum(counts)
    x, xs = fp8_rows(g, n, 384)
    w, ws = fp8_weights(g, len(counts), 256, 384)
    x.view(torch.uint8)[0], xs[0] = 0, 0.0
    off = offsets_of(counts)
    y, ys = torch.ones(n, 256, device="cuda").to(E4M3), torch.ones(n, 2, device="cuda")
    ep.ep_expert_fp8(x, xs, w, ws, y, expert_offsets=off, y_scales=ys)
    assert (y[0].float() == 0).all() and (ys[0] == 0).all()
    for sx, sw in ((2.0 ** 60, 2.0 ** 55), (2.0 ** -60, 2.0 ** -50), (2.0 ** 100, 2.0 ** -90)):
        spread = torch.tensor([1.0, 2.0 ** -20, 2.0 ** 9], device="cuda")
        y = torch.empty(n, 256, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_fp8(x, xs * sx * spread, w, ws * sw, y, expert_offsets=off)
        want, tol = fp8_reference(counts, x, xs * sx * spread, w, ws * sw, False)
        assert want.abs().max() < 3e38
        within(y, want, tol + U[y.dtype] * want.abs() + 2.0 ** -134)


@pytest.mark.parametrize("grad_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", [[5, 0, 130], [0, 0, 1]])
def test_accumulated_weight_gradients(ep, grad_dtype, counts):
    H, F, n, E, g = 72, 40, sum(counts), 3, gen(4)
    x, up, down = block_inputs(g, counts, H, F, torch.bfloat16)
    gate_up, act, dy = (randn(g, n, k, dtype=torch.bfloat16) for k in (2 * F, F, H))
    before = [randn(g, E, 2 * F, H, dtype=grad_dtype), randn(g, E, H, F, dtype=grad_dtype)]
    dgu, off = torch.empty_like(gate_up), offsets_of(counts)

    def call(grads, accumulate):
        ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, dgu, None, *grads, expert_offsets=off, accumulate=accumulate)
        return grads

    alone = call([torch.empty_like(t, dtype=torch.float32) for t in before], False)
    both = call([t.clone() for t in before], True)
    for a, b, c in zip(alone, before, both):
        want = a.double() + b.double()
        within(c, want, (U[grad_dtype] + U[torch.float32]) * want.abs() + U[torch.float32] * b.double().abs())


def test_parts_of_the_block_alone(ep):
    """act without y; each gradient without the others; no rows at all."""
    counts, H, F = [7, 0, 140], 72, 40
    g, n, off = gen(6), sum(counts), offsets_of(counts)
    x, up, down = block_inputs(g, counts, H, F, torch.float16)
    act, y, alone = (torch.empty(n, k, dtype=torch.float16, device="cuda") for k in (F, H, F))
    ep.ep_expert_ffn(x, up, down, act, y, expert_offsets=off)
    ep.ep_expert_ffn(x, up, None, alone, None, expert_offsets=off)
    assert torch.equal(act, alone)
    gate_up, dy = randn(g, n, 2 * F, dtype=torch.float16), randn(g, n, H, dtype=torch.float16)

    def call(dx=None, dup=None, ddown=None):
        dgu = torch.empty_like(gate_up)
        ep.ep_expert_ffn_backward(dy, None if dup is None else x, gate_up, None if ddown is None else act, None if dx is None else up, down,
                                  dgu, dx, dup, ddown, expert_offsets=off)
        return dgu

    full = [torch.empty_like(t) for t in (x, up, down)]
    dgu = call(*full)
    assert torch.equal(call(), dgu)
    for k in range(3):
        part = [torch.empty_like(t) if i == k else None for i, t in enumerate(full)]
        assert torch.equal(call(*part), dgu) and torch.equal(part[k], full[k])
    none = torch.empty(0, H, dtype=torch.float16, device="cuda")
    dup, ddown = torch.full_like(up, math.nan), torch.full_like(down, math.nan)
    ep.ep_expert_ffn_backward(none, none, none.new_empty(0, 2 * F), none.new_empty(0, F), up, down, none.new_empty(0, 2 * F), none, dup, ddown,
                              expert_offsets=offsets_of([0, 0, 0]))
    assert (dup == 0).all() and (ddown == 0).all()


def test_repeated_calls_give_the_same_bits(ep):
    counts, H, F = [64, 1, 300, 0, 40], 264, 136
    g, n, off = gen(8), sum(counts), offsets_of(counts)
    x, up, down = block_inputs(g, counts, H, F, torch.bfloat16)
    gate_up, act, dy = (randn(g, n, k, dtype=torch.bfloat16) for k in (2 * F, F, H))
    x8, xs = fp8_rows(g, n, 512)
    w, ws = fp8_weights(g, 5, 256, 512)

    def call():
        outs = [torch.empty(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H, 2 * F, H, 256)] + [torch.empty_like(up), torch.empty_like(down)]
        ep.ep_expert_ffn(x, up, down, outs[0], outs[1], expert_offsets=off)
        ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, outs[2], outs[3], outs[5], outs[6], expert_offsets=off)
        ep.ep_expert_fp8(x8, xs, w, ws, outs[4], expert_offsets=off)
        return outs

    first = call()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))


@pytest.mark.parametrize("rows", [1, 2, 5, 16, 17, 31, 32, 33, 48, 64, 65, 127, 128, 129, 256, 257, 300])
@pytest.mark.parametrize("swiglu", [False, True])
def test_fp8_one_matrix_of_any_number_of_rows(ep, rows, swiglu):
    """Without offsets; few items are shared by the CTAs of clusters."""
    g, I, O = gen(rows), 1152, 384
    x, xs = fp8_rows(g, rows, I)
    w, ws = fp8_weights(g, 1, O, I)
    for dtype in (torch.bfloat16, E4M3):
        cols = O // 2 if swiglu else O
        if dtype == E4M3 and cols % 128:
            continue
        y = torch.empty(rows, cols, device="cuda").to(dtype)
        ys = torch.empty(rows, cols // 128, device="cuda")
        ep.ep_expert_fp8(x, xs, w, ws, y, activation=ep.EP_ACT_SWIGLU if swiglu else ep.EP_ACT_NONE, y_scales=ys if dtype == E4M3 else None)
        want, tol = fp8_reference([rows], x, xs, w, ws, swiglu)
        if dtype == E4M3:
            wide = ys.double().repeat_interleave(128, 1)
            within(y.double() * wide, want, tol + (want.abs() + tol) * 2.0 ** -4 + 2.0 ** -10 * wide)
        else:
            within(y, want, tol + U[dtype] * want.abs())


@pytest.mark.parametrize("rows", [1, 8, 9, 63, 64, 65, 128, 255, 256, 257, 513])
def test_block_of_one_expert(ep, rows):
    x, up, down, act, y = one_block(ep, [rows], 328, 264)
    check_block_rows(x, up, down, act, y, [0] * rows)


def test_past_32_bit_offsets(ep):
    """Weights of more than 2^31 elements, and rows that far apart."""
    E, O, I = 34, 8192, 8192                       # 2.28e9 codes
    g = gen(2)
    w = torch.zeros(E, O, I, dtype=torch.uint8, device="cuda").view(E4M3)
    ws = torch.ones(E, O // 128, I // 128, device="cuda")
    rows = torch.randint(0, O, (E, 4), generator=g)
    one = torch.randn(E, 4, I, generator=g).to(E4M3).cuda()
    for e in range(E):
        w[e].view(torch.uint8)[rows[e].cuda()] = one[e].view(torch.uint8)
    x, xs = fp8_rows(g, E, I)
    y = torch.empty(E, O, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_fp8(x, xs, w, ws, y, expert_offsets=offsets_of([1] * E))
    xd = decoded(x, xs)
    for e in range(E):
        want, size = one[e].double() @ xd[e], one[e].double().abs() @ xd[e].abs()
        within(y[e][rows[e].cuda()], want, (128 + 4 + I // 128) * F32 * size + U[y.dtype] * want.abs())
    assert (y != 0).sum() <= 4 * E
    del w
    n, far = 3, 1 << 30                            # rows 2^30 elements apart
    H, F = 64, 32
    base = torch.zeros(2 * far + H, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((n, H), (far, 1))
    x.copy_(randn(g, n, H))
    up, down = randn(g, 1, 2 * F, H, dtype=torch.bfloat16, scale=0.1), randn(g, 1, H, F, dtype=torch.bfloat16, scale=0.1)
    outs = [[torch.empty(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H)] for _ in range(2)]
    ep.ep_expert_ffn(x, up, down, *outs[0])
    ep.ep_expert_ffn(x.contiguous(), up, down, *outs[1])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    wide = torch.empty(2 * far + H, dtype=torch.bfloat16, device="cuda").as_strided((n, H), (far, 1))
    ep.ep_expert_ffn(x, up, down, outs[0][0], wide)
    assert torch.equal(wide, outs[1][1])


def test_weight_gradients_past_32_bit_offsets(ep):
    E, H, F = 17, 8192, 8192                       # a gradient of 2.28e9 elements
    g = gen(7)
    down = torch.zeros(E, H, F, dtype=torch.bfloat16, device="cuda")
    gate_up, act, dy = randn(g, E, 2 * F, dtype=torch.bfloat16), randn(g, E, F, dtype=torch.bfloat16), randn(g, E, H, dtype=torch.bfloat16)
    dgu, dw = torch.empty_like(gate_up), torch.empty(2 * E, H, F, dtype=torch.bfloat16, device="cuda")[:E]
    ep.ep_expert_ffn_backward(dy, None, gate_up, act, None, down, dgu, grad_w_down=dw, expert_offsets=offsets_of([1] * E))
    for e in range(E):
        want = (dy[e].float()[:, None] * act[e].float()).bfloat16()   # one product, rounded once
        assert torch.equal(dw[e], want)


# ------------------------------------------------------------------ streams, graphs, and all together

def test_on_another_stream_and_in_a_graph(ep):
    counts, H, F = [17, 0, 200, 40], 136, 128
    g, n = gen(11), sum(counts)
    x, up, down = block_inputs(g, counts, H, F, torch.bfloat16)
    gate_up, act, dy = (randn(g, n, k, dtype=torch.bfloat16) for k in (2 * F, F, H))
    x8, xs = fp8_rows(g, n, 256)
    w, ws = fp8_weights(g, 4, 256, 256)
    off = offsets_of(counts)
    outs = [torch.zeros(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H, 2 * F, H)] + [torch.zeros_like(up), torch.zeros_like(down)]
    q, qs = torch.zeros(n, 128, device="cuda").to(E4M3), torch.zeros(n, 1, device="cuda")

    def call(stream=None):
        ep.ep_expert_ffn(x, up, down, outs[0], outs[1], expert_offsets=off, stream=stream)
        ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, outs[2], outs[3], outs[4], outs[5], expert_offsets=off, stream=stream)
        ep.ep_expert_fp8(x8, xs, w, ws, q, expert_offsets=off, y_scales=qs, activation=ep.EP_ACT_SWIGLU, stream=stream)

    def taken():
        torch.cuda.synchronize()
        got = [t.clone() for t in outs + [q.view(torch.uint8), qs]]
        for t in outs + [q.view(torch.uint8), qs]:
            t.zero_()
        torch.cuda.synchronize()
        return got

    call()
    want = taken()
    side = torch.cuda.Stream()
    call(side)
    assert all(torch.equal(a, b) for a, b in zip(want, taken()))
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, taken()))
    # new routing, same graph: what was a row of one expert is another's now
    new = [200, 17, 40, 0]
    off.copy_(offsets_of(new))
    graph.replay()
    replayed = taken()
    call()
    assert all(torch.equal(a, b) for a, b in zip(replayed, taken()))
    check_block_rows(x, up, down, replayed[0], replayed[1], [e for e, m in enumerate(new) for _ in range(m)])


def test_two_streams_at_once(ep):
    """Calls of the same operators that overlap on the GPU do not disturb each other."""
    g = gen(12)
    jobs = []
    for k in range(2):
        counts = [30 + 100 * k, 0, 250]
        x, up, down = block_inputs(g, counts, 264, 136, torch.bfloat16)
        jobs.append((x, up, down, offsets_of(counts), [torch.empty(sum(counts), w, dtype=torch.bfloat16, device="cuda") for w in (136, 264)]))
    for x, up, down, off, outs in jobs:
        ep.ep_expert_ffn(x, up, down, *outs, expert_offsets=off)
    want = [[t.clone() for t in j[4]] for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (x, up, down, off, outs) in zip(streams, jobs):
            ep.ep_expert_ffn(x, up, down, *outs, expert_offsets=off, stream=s)
    torch.cuda.synchronize()
    for j, w in zip(jobs, want):
        assert all(torch.equal(a, b) for a, b in zip(j[4], w))


def test_fp8_rows_of_the_dispatch(ep):
    """Layout, fp8 dispatch in every scale mode, both products, weighted combine: one serving step of a layer."""
    T, H, F, E, K = 100, 256, 128, 16, 4
    g = gen(13)
    x = randn(g, T, H, dtype=torch.bfloat16)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :K].cuda()
    wt = torch.rand(T, K, generator=g).cuda()
    up, ups = fp8_weights(g, E, 2 * F, H)
    down, downs = fp8_weights(g, E, H, F)
    cnt, ntr, itr, off = (torch.empty(s, dtype=d, device="cuda") for s, d in (((E,), torch.int32), ((1,), torch.int32), ((T, 1), torch.uint8), ((E + 1,), torch.int32)))
    h = ep.ep_layout(idx, E, 1, cnt, ntr, itr, off)
    n = T * K
    for mode in (0, 1, 2):
        q = torch.empty(n, H, dtype=torch.uint8, device="cuda")
        s = torch.empty(H // 128, n, dtype=torch.uint8 if mode == 2 else torch.float32, device="cuda")
        ep.ep_dispatch_ex(h, x, q, n, recv_scales=s, out_dtype=ep.EP_DTYPE_FP8_E4M3, scale_mode=mode, scales_col_major=True, scales_ld=n)
        act, acts = torch.empty(n, F, device="cuda").to(E4M3), torch.empty(n, F // 128, dtype=s.dtype, device="cuda")
        y, out = torch.empty(n, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_fp8(q.view(E4M3), s.t(), up, ups, act, expert_offsets=off, y_scales=acts, scale_mode=mode, activation=ep.EP_ACT_SWIGLU)
        ep.ep_expert_fp8(act, acts, down, downs, y, expert_offsets=off)
        ep.ep_combine(h, y, out, topk_weights=wt)
        # the layer in 64 bits from the bf16 tokens: two roundings to 8 bits lie between, half a step of 2^-4 of each value
        full = torch.zeros(T, H, dtype=torch.float64)
        scale = torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for k in range(K):
                e = int(idx[t, k])
                w1 = up[e].double() * ups[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
                w2 = down[e].double() * downs[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
                xv = x[t].double()
                a, tol = silu_parts((w1 @ xv)[None], 2.0 ** -4 * (w1.abs() @ xv.abs())[None])
                full[t] += float(wt[t, k]) * (w2 @ a[0]).cpu()
                scale[t] += float(wt[t, k]) * (w2.abs() @ (tol[0] + 2.0 ** -4 * (a[0].abs() + tol[0]) + 2.0 ** -9 * a[0].abs().max())).cpu()
        within(out, full, scale + 2.0 ** -7 * (scale + full.abs()))
    h.destroy()


def test_training_step_against_autograd(ep):
    """Layout, dispatch, block, combine and all of it backwards, against 64-bit autograd of the same layer."""
    T, H, F, E, K = 90, 128, 72, 8, 2
    g = gen(14)
    x = randn(g, T, H, dtype=torch.bfloat16)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :K].cuda()
    wt = torch.rand(T, K, generator=g).cuda()
    up, down = randn(g, E, 2 * F, H, dtype=torch.bfloat16, scale=H ** -0.5), randn(g, E, H, F, dtype=torch.bfloat16, scale=F ** -0.5)
    d_out = randn(g, T, H, dtype=torch.bfloat16)
    cnt, ntr, itr, off = (torch.empty(s, dtype=d, device="cuda") for s, d in (((E,), torch.int32), ((1,), torch.int32), ((T, 1), torch.uint8), ((E + 1,), torch.int32)))
    h = ep.ep_layout(idx, E, 1, cnt, ntr, itr, off)
    n, bf16 = T * K, dict(dtype=torch.bfloat16, device="cuda")
    recv, act, y, gate_up, out = (torch.empty(n, k, **bf16) for k in (H, F, H, 2 * F, H))
    out = torch.empty(T, H, **bf16)
    ep.ep_dispatch_ex(h, x, recv, n, out_dtype=ep.EP_DTYPE_BF16)
    ep.ep_expert_ffn(recv, up, down, act, y, gate_up=gate_up, expert_offsets=off)
    ep.ep_combine(h, y, out, topk_weights=wt)
    dy, d_wt, dgu, d_recv, dx = torch.empty(n, H, **bf16), torch.empty(T, K, device="cuda"), torch.empty(n, 2 * F, **bf16), torch.empty(n, H, **bf16), torch.empty(T, H, **bf16)
    d_up, d_down = torch.empty(E, 2 * F, H, device="cuda"), torch.empty(E, H, F, device="cuda")
    ep.ep_combine_backward(h, d_out, y, grad_y=dy, topk_weights=wt, grad_topk_weights=d_wt)
    ep.ep_expert_ffn_backward(dy, recv, gate_up, act, up, down, dgu, d_recv, d_up, d_down, expert_offsets=off)
    ep.ep_dispatch_backward(h, d_recv, dx)
    h.destroy()
    leaves = [t.double().requires_grad_() for t in (x, up, down, wt)]
    X, W1, W2, W = leaves
    hidden = torch.einsum("tkfh,th->tkf", W1[idx], X)
    a = torch.nn.functional.silu(hidden[..., :F]) * hidden[..., F:]
    result = (torch.einsum("tkhf,tkf->tkh", W2[idx], a) * W[..., None]).sum(1)
    (result * d_out.double()).sum().backward()
    # each of the 16-bit tensors on the way (at most five) is off by 2^-8 of its values, at random: 5 * 2^-8 of the result's norm
    for got, want in ((out, result.detach()), (dx, X.grad), (d_up, W1.grad), (d_down, W2.grad), (d_wt, W.grad)):
        assert (got.double() - want).norm() <= 5 * 2.0 ** -8 * want.norm()


def test_gradients_against_differences(ep):
    """The library's own forward, moved by small steps: the difference of a linear loss is the gradient along the step."""
    counts, H, F = [40, 0, 25], 64, 48
    n, off, g = sum(counts), offsets_of(counts), gen(15)
    x, up, down = block_inputs(g, counts, H, F, torch.float16)
    d = randn(g, n, H, dtype=torch.float16)

    def loss(x, up, down):
        act, y, gate_up = (torch.empty(n, k, dtype=torch.float16, device="cuda") for k in (F, H, 2 * F))
        ep.ep_expert_ffn(x, up, down, act, y, gate_up=gate_up, expert_offsets=off)
        return (y.double() * d.double()).sum().item(), act, gate_up

    _, act, gate_up = loss(x, up, down)
    dgu, dx, dup, ddown = torch.empty_like(gate_up), torch.empty_like(x), torch.empty_like(up, dtype=torch.float32), torch.empty_like(down, dtype=torch.float32)
    ep.ep_expert_ffn_backward(d, x, gate_up, act, up, down, dgu, dx, dup, ddown, expert_offsets=off)
    for k, (t, grad) in enumerate(((x, dx), (up, dup), (down, ddown))):
        step = (torch.sign(grad.double()) * 2.0 ** -6 * t.double().abs().mean()).to(torch.float16)
        moved = [[u.clone() for u in (x, up, down)] for _ in range(2)]
        moved[0][k] += step
        moved[1][k] -= step
        real = (moved[0][k].double() - moved[1][k].double())
        got = loss(*moved[0])[0] - loss(*moved[1])[0]
        want = (real * grad.double()).sum().item()
        # y's rounding (2^-11 of each term, at random over n H terms) against a difference that is 2^-6 of the loss's scale,
        # and the third-order term of a step of 2^-6
        noise = 2 * 2.0 ** -11 * 6 * (n * H) ** 0.5 * H ** 0.5
        assert abs(got - want) <= 0.02 * abs(want) + noise, (k, got, want, noise)


def test_train_experts_example(ep):
    """The example's layer on two micro-batches against 64-bit autograd of the same layer, routing taken from the example."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_experts
    T, H, F, E, K = 70, 128, 72, 8, 3
    layer = train_experts.ExpertLayer(T, hidden=H, inner=F, experts=E, topk=K)
    g = gen(16)
    gate, w1, w2 = (t.double().requires_grad_() for t in (layer.gate, layer.up16, layer.down16))
    for k in range(2):
        x, d_out = randn(g, T, H, dtype=torch.bfloat16), randn(g, T, H, dtype=torch.bfloat16)
        out = layer.forward(x).clone()
        dx = layer.backward(d_out, add=k > 0)
        X = x.double().requires_grad_()
        top = torch.softmax((X @ gate.t()).gather(1, layer.idx), 1)
        hidden = torch.einsum("tkfh,th->tkf", w1[layer.idx], X)
        a = torch.nn.functional.silu(hidden[..., :F]) * hidden[..., F:]
        result = (torch.einsum("tkhf,tkf->tkh", w2[layer.idx], a) * top[..., None]).sum(1)
        (result * d_out.double()).sum().backward()
        # as above, and dx is the sum of two rounded parts
        for got, want in ((out, result.detach()), (dx, X.grad)):
            assert (got.double() - want).norm() <= 6 * 2.0 ** -8 * want.norm()
    for got, want in ((layer.grad_gate, gate.grad), (layer.grad_up, w1.grad), (layer.grad_down, w2.grad)):
        assert (got.double() - want).norm() <= 5 * 2.0 ** -8 * want.norm()
    before = layer.w_up.clone()
    layer.step(0.5)
    assert torch.equal(layer.w_up, before - 0.5 * layer.grad_up) and torch.equal(layer.up16, layer.w_up.bfloat16())
    layer.handle.destroy()


def test_train_experts_example_runs_as_a_program():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "train_experts.py"), "--tokens", "96", "--steps", "3",
                        "--hidden", "256", "--inner", "128"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "gradients finite: True" in r.stdout


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_fp8_odd_output_rows_of_full_and_short_tiles(ep, late, dtype):
    """Outputs whose rows start anywhere, experts of full tiles beside short ones, so that a CTA has both in turn."""
    counts = [128 + 3 * k % 50 if k % 3 else 200 - 7 * (k % 9) for k in range(40)]
    I, O, n = 256, 515, sum(counts)
    g = gen(17)
    x, xs = fp8_rows(g, n, I)
    w, ws = fp8_weights(g, len(counts), O, I)
    wide = torch.full((n, O + 6), math.nan, dtype=dtype, device="cuda")
    y = wide[:, 3:3 + O] if late else wide[:, :O]
    ep.ep_expert_fp8(x, xs, w, ws, y, expert_offsets=offsets_of(counts))
    want, tol = fp8_reference(counts, x, xs, w, ws, False)
    within(y, want, tol + U[dtype] * want.abs() + TINY[dtype])
    assert wide[:, 3 + O if late else O:].isnan().all() and (not late or wide[:, :3].isnan().all())


def test_experts_without_rows_keep_accumulated_gradients(ep):
    """With accumulate an expert without rows keeps what is there, to the bit."""
    counts, H, F = [0, 33, 0, 5], 136, 40
    n, g = sum(counts), gen(18)
    x, up, down = block_inputs(g, counts, H, F, torch.bfloat16)
    act, y, gate_up = (torch.empty(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H, 2 * F))
    off = offsets_of(counts)
    ep.ep_expert_ffn(x, up, down, act, y, gate_up=gate_up, expert_offsets=off)
    for dtype in (torch.bfloat16, torch.float32):
        d_up, d_down = randn(g, 4, 2 * F, H, dtype=dtype), randn(g, 4, H, F, dtype=dtype)
        d_up[0, 0, :3] = torch.tensor([-0.0, math.inf, math.nan])
        old = d_up.clone(), d_down.clone()
        ep.ep_expert_ffn_backward(y, x, gate_up, act, up, down, torch.empty_like(gate_up), torch.empty_like(x), d_up, d_down,
                                  expert_offsets=off, accumulate=True)
        bits = torch.int32 if dtype == torch.float32 else torch.int16
        for got, was in zip((d_up, d_down), old):
            assert torch.equal(got[[0, 2]].view(bits), was[[0, 2]].view(bits))
            assert not torch.equal(got[1], was[1]) and not torch.equal(got[3], was[3])


@pytest.mark.parametrize("counts,I,O", [([5447], 128, 1030), ([138] * 60, 128, 700), ([300, 0, 777, 65, 1025, 90, 131] * 6, 256, 1290)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_fp8_every_tile_has_its_turn(ep, counts, I, O, swiglu):
    """More tiles than CTAs, several of an expert, at every place against the number of CTAs: all rows are written."""
    run_fp8(ep, counts, I, O, swiglu)


@pytest.mark.parametrize("counts", [[1, 40], [300, 0, 129], [20] * 30])
@pytest.mark.parametrize("H,F", [(64, 72), (264, 520)])
def test_gradients_in_place(ep, counts, H, F):
    """grad_gate_up may take the place of gate_up, and grad_x that of grad_y: the same bits as apart."""
    g, n, off = gen(19), sum(counts), offsets_of(counts)
    x, up, down = block_inputs(g, counts, H, F, torch.bfloat16)
    act, y, gate_up = (torch.empty(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H, 2 * F))
    ep.ep_expert_ffn(x, up, down, act, y, gate_up=gate_up, expert_offsets=off)
    dy = randn(g, n, H, dtype=torch.bfloat16)
    dgu, dx, dup, ddown = (torch.full_like(t, math.nan) for t in (gate_up, x, up, down))
    ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, dgu, dx, dup, ddown, expert_offsets=off)
    dup2, ddown2 = torch.full_like(up, math.nan), torch.full_like(down, math.nan)
    ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, gate_up, dy, dup2, ddown2, expert_offsets=off)
    for got, want in ((gate_up, dgu), (dy, dx), (dup2, dup), (ddown2, ddown)):
        assert torch.equal(got, want)


def test_in_a_captured_step_twice(ep):
    """A captured forward and backward between which an eager call runs on other buffers, replayed several times."""
    counts, H, F = [70, 3, 0, 190], 136, 88
    g, n, off = gen(20), sum(counts), offsets_of(counts)

    def buffers():
        x, up, down = block_inputs(g, counts, H, F, torch.bfloat16)
        outs = [torch.empty(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H, 2 * F, 2 * F, H)]
        return x, up, down, outs, torch.zeros(4, 2 * F, H, device="cuda"), torch.zeros(4, H, F, device="cuda")

    def step(x, up, down, outs, dup, ddown):
        act, y, gate_up, dgu, dx = outs
        ep.ep_expert_ffn(x, up, down, act, y, gate_up=gate_up, expert_offsets=off)
        ep.ep_expert_ffn_backward(y, x, gate_up, act, up, down, dgu, dx, dup, ddown, expert_offsets=off, accumulate=True)

    one, two = buffers(), buffers()
    step(*one)
    step(*two)
    want = [t.clone() for t in one[3]] + [one[4].clone(), one[5].clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*one)
    for t in one[3]:
        t.fill_(math.nan)
    one[4].zero_()
    one[5].zero_()
    for _ in range(2):
        graph.replay()
        step(*two)
    for got, w in zip(one[3], want):
        assert torch.equal(got, w)
    # the same fp32 gradient added twice is its double, exactly
    assert torch.equal(one[4], 2 * want[5]) and torch.equal(one[5], 2 * want[6])
