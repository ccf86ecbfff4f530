"""The experts' products at sizes that take the larger tiles: every shape of the kernels, beside one another in a call."""
import math

import pytest
import torch

import test_gpu_experts as plain

from test_gpu_experts import E4M3, E5M2, F32, TINY, U, ep, fp8_reference, fp8_rows, fp8_weights, gen, offsets_of, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("I", [128, 256, 640, 1152])
@pytest.mark.parametrize("swiglu", [False, True])
def test_fp8_short_tiles_behind_full_ones(ep, I, swiglu):
    """Experts of a full tile and a short one, more tiles than CTAs: a CTA's sums of a short tile follow a full tile's in the
    same buffers, at every place in their turn. Right, and the same bits each time."""
    counts = [128 + 1 + 13 * k % 64 for k in range(48)]
    n, O, g = sum(counts), 1280, gen(I)
    x, xs = fp8_rows(g, n, I)
    w, ws = fp8_weights(g, len(counts), O, I)
    off = offsets_of(counts)

    def call():
        y = torch.full((n, O // 2 if swiglu else O), math.nan, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_fp8(x, xs, w, ws, y, expert_offsets=off, activation=ep.EP_ACT_SWIGLU if swiglu else ep.EP_ACT_NONE)
        return y

    first = call()
    want, tol = fp8_reference(counts, x, xs, w, ws, swiglu)
    within(first, want, tol + U[first.dtype] * want.abs() + TINY[first.dtype])
    for _ in range(20):
        assert torch.equal(call(), first)


# ------------------------------------------------------------------ which tiles a call takes

def most_tiles(counts, cap):
    rows, used = sum(counts), min(sum(counts), len(counts))
    return (rows + used * (cap - 1)) // cap


def mean_rows(counts):
    return (sum(counts) - 1) // min(sum(counts), len(counts)) + 1


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def fp8_tiles(counts, O, swiglu):
    """The library's rule: 32 or 64 rows as columns, or "lanes"."""
    cols = O // 2 if swiglu else O
    m_tiles = -(-cols // (128 if swiglu else 256))
    few = lambda cap, times: times * most_tiles(counts, cap) * m_tiles <= sms()
    if mean_rows(counts) <= 24 or few(64, 2):
        return 32
    return 64 if mean_rows(counts) <= 48 or few(128, 3) or (swiglu and cols % 64) else "lanes"


def block_tiles(counts, channels, of_tile):
    """The library's rule: rows of a tile of the 16-bit products, at most."""
    mean = mean_rows(counts)
    cap = 32 if mean <= 24 else 64 if mean <= 48 else 128 if mean <= 112 else 256
    while cap > 32 and 4 * most_tiles(counts, cap) * -(-channels // of_tile) <= sms():
        cap //= 2
    return cap


# ------------------------------------------------------------------ fp8

FP8_COUNTS = {64: [25 + 7 * k % 37 for k in range(40)] + [64, 65, 1, 0],      # (tiles of nearly equal rows)
              "lanes": [60 + 97 * k % 240 for k in range(40)] + [128, 129, 64, 65, 192, 193, 1, 0]}
TILES = pytest.mark.parametrize("tiles", [64, "lanes"])


def fp8_case(tiles, I, O, swiglu, x_dtype=E4M3, ue8m0=False, columns=False):
    counts = FP8_COUNTS[tiles]
    assert fp8_tiles(counts, O, swiglu) == tiles
    g = gen(I + O)
    x, xs = fp8_rows(g, sum(counts), I, x_dtype, ue8m0, columns)
    return counts, x, xs, *fp8_weights(g, len(counts), O, I)


def apart(n, cols, dtype, extra):
    """[n + 1, cols] of 7 in rows `extra` further apart, and the whole."""
    whole = torch.full((n + 1, cols + extra), 7.0, device="cuda").to(dtype)
    return whole[:, :cols], whole


def others_kept(y, whole, cols):
    raw = whole.view(torch.uint8) if whole.dtype == E4M3 else whole
    seven = torch.tensor(7.0).to(whole.dtype).view(raw.dtype).item() if whole.dtype == E4M3 else 7.0
    assert (raw[:, cols:] == seven).all() and (raw[-1] == seven).all()


@TILES
@pytest.mark.parametrize("O", [640, 1024])   # (with the activation 320 channels: up rows of one tile lie in two blocks of scales)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("extra", [0, 5])
def test_fp8_outputs_of_large_tiles(ep, tiles, O, swiglu, dtype, extra):
    counts, x, xs, w, ws = fp8_case(tiles, 384, O, swiglu)
    cols = O // 2 if swiglu else O
    y, whole = apart(len(x), cols, dtype, extra)
    ep.ep_expert_fp8(x, xs, w, ws, y[:-1], expert_offsets=offsets_of(counts), activation=int(swiglu))
    want, tol = fp8_reference(counts, x, xs, w, ws, swiglu)
    within(y[:-1], want, tol + U[dtype] * want.abs() + TINY[dtype])
    others_kept(y, whole, cols)


@TILES
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("x_dtype", [E4M3, E5M2])
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("columns", [False, True])
def test_fp8_row_formats_of_large_tiles(ep, tiles, swiglu, x_dtype, ue8m0, columns):
    counts, x, xs, w, ws = fp8_case(tiles, 640, 768, swiglu, x_dtype, ue8m0, columns)
    y = torch.full((len(x), 384 if swiglu else 768), math.nan, dtype=torch.float16, device="cuda")
    ep.ep_expert_fp8(x, xs, w, ws, y, expert_offsets=offsets_of(counts), activation=int(swiglu))
    want, tol = fp8_reference(counts, x, xs, w, ws, swiglu)
    within(y, want, tol + U[y.dtype] * want.abs() + TINY[y.dtype])


@TILES
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("extra,columns", [(0, False), (16, True), (3, False)])
def test_fp8_quantised_outputs_of_large_tiles(ep, tiles, swiglu, mode, extra, columns):
    cols = 640
    counts, x, xs, w, ws = fp8_case(tiles, 384, 2 * cols if swiglu else cols, swiglu)
    n, kind = len(x), torch.uint8 if mode == 2 else torch.float32
    y, whole = apart(n, cols, E4M3, extra)
    ys = torch.zeros(cols // 128, n, dtype=kind, device="cuda").t() if columns else torch.zeros(n, cols // 128, dtype=kind, device="cuda")
    ep.ep_expert_fp8(x, xs, w, ws, y[:-1], expert_offsets=offsets_of(counts), y_scales=ys, scale_mode=mode, activation=int(swiglu))
    want, tol = (t.cpu() for t in fp8_reference(counts, x, xs, w, ws, swiglu))
    s = torch.exp2(ys.double() - 127).cpu() if mode == 2 else ys.double().cpu()
    blocks, block_tol = want.abs().view(n, -1, 128).amax(2) / 448, tol.view(n, -1, 128).amax(2) / 448
    if mode == 0:
        within(s, blocks, block_tol + U[torch.float32] * blocks)
    else:   # the smallest power of two that is not below amax / 448, with what that may be off by
        assert torch.equal(torch.exp2(torch.round(torch.log2(s))), s)
        assert (s >= (blocks - block_tol) * (1 - F32)).all() and (s < 2 * (blocks + block_tol) * (1 + F32)).all()
    wide = s.repeat_interleave(128, 1)
    # a code is off by half a step: 2^-4 of it, or half of the smallest step, 2^-10
    within(y[:-1].double().cpu() * wide, want, tol + (want.abs() + tol) * 2.0 ** -4 + 2.0 ** -10 * wide)
    others_kept(y, whole, cols)


@TILES
@pytest.mark.parametrize("swiglu", [False, True])
def test_fp8_nan_stays_in_its_row_of_large_tiles(ep, tiles, swiglu):
    counts, x, xs, w, ws = fp8_case(tiles, 384, 768, swiglu)
    off, n, cols = offsets_of(counts), len(x), 384 if swiglu else 768
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[::11] = True
    bad[off[1:-1].long().clamp(max=n - 1)] = True    # first rows of experts, behind the last of others
    codes, scales = x.clone(), xs.clone()
    codes.view(torch.uint8)[::11, 200] = 0x7F
    scales[bad, 1] = math.nan
    outs = []
    for c, s in ((x, xs), (codes, scales)):
        y = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
        q, qs = torch.empty(n, cols, device="cuda").to(E4M3), torch.empty(n, cols // 128, device="cuda")
        for out, out_scales in ((y, None), (q, qs)):
            ep.ep_expert_fp8(c, s, w, ws, out, expert_offsets=off, y_scales=out_scales, activation=int(swiglu))
        outs.append((y, q.float(), qs))
    for clean, dirty in zip(*outs):
        assert torch.equal(clean[~bad], dirty[~bad]) and dirty[bad].isnan().all()


# ------------------------------------------------------------------ gated block

BLOCK_COUNTS = {64: [25 + 7 * k % 37 for k in range(40)] + [64, 65, 1, 0], 128: [60 + 7 * k % 51 for k in range(30)] + [128, 129, 257, 1, 0],
                256: [130 + 97 * k % 571 for k in range(20)] + [256, 257, 3, 0], "wraps": [5, 4500, 300]}   # (more than 16 tiles of an expert)
CAPS = pytest.mark.parametrize("cap", list(BLOCK_COUNTS))


def block_case(cap, H, F):
    """Counts for which all four products that have rows as columns take tiles of at most `cap` rows."""
    counts = BLOCK_COUNTS[cap]
    for channels, of_tile in ((F, 128), (H, 256), (F, 256)):
        assert block_tiles(counts, channels, of_tile) == (256 if cap == "wraps" else cap)
    return counts


@CAPS
@pytest.mark.parametrize("H,F", [(1032, 1032), (776, 1288)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_block_of_large_tiles(ep, cap, H, F, dtype):
    plain.test_block(ep, block_case(cap, H, F), H, F, dtype)


@CAPS
@pytest.mark.parametrize("H,F", [(1032, 1032), (776, 1288)])
@pytest.mark.parametrize("dtype,grad_dtype", [(torch.bfloat16, torch.float32), (torch.float16, torch.float16)])
def test_block_backward_of_large_tiles(ep, cap, H, F, dtype, grad_dtype):
    plain.test_block_backward(ep, block_case(cap, H, F), H, F, dtype, grad_dtype)


@CAPS
def test_gradients_in_place_of_large_tiles(ep, cap):
    plain.test_gradients_in_place(ep, block_case(cap, 1032, 1032), 1032, 1032)


@pytest.mark.parametrize("counts,cap", [([40, 33] + [45] * 60, 64), ([100, 90] + [100] * 30, 128), ([300, 260, 20000], 256)])
def test_nan_and_infinity_stay_in_their_rows_of_large_tiles(ep, counts, cap):
    """The second expert has a row of NaN, the third infinite weights: the other rows and experts keep their bits."""
    H, F, n, off, g = 136, 72, sum(counts), offsets_of(counts), gen(22)
    assert {block_tiles(counts, H, 256), block_tiles(counts, F, 128), block_tiles(counts, F, 256)} == {cap}
    x, up, down = plain.block_inputs(g, counts, H, F, torch.bfloat16)
    gate_up, act, dy = (plain.randn(g, n, k, dtype=torch.bfloat16) for k in (2 * F, F, H))

    def all_of(x, up, down, gate_up, act, dy):
        outs = [torch.empty(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H, 2 * F, 2 * F, H)]
        grads = [torch.empty_like(up), torch.empty_like(down)]
        ep.ep_expert_ffn(x, up, down, outs[0], outs[1], gate_up=outs[2], expert_offsets=off)
        ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, outs[3], outs[4], *grads, expert_offsets=off)
        return outs, grads

    clean = all_of(x, up, down, gate_up, act, dy)
    bad = [t.clone() for t in (x, up, down, gate_up, act, dy)]
    first, third = counts[0], counts[0] + counts[1]
    for t in (bad[0], bad[3], bad[4], bad[5]):
        t[first] = math.nan
    bad[1][2], bad[2][2] = math.inf, math.inf
    dirty = all_of(*bad)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[first] = False
    keep[third:third + counts[2]] = False
    for a, b in zip(clean[0], dirty[0]):
        assert torch.equal(a[keep], b[keep]) and b[first].isnan().any()
    others = [e for e in range(len(counts)) if e not in (1, 2)]
    for a, b in zip(clean[1], dirty[1]):
        assert torch.equal(a[others], b[others]) and b[1].isnan().any()


@CAPS
def test_strided_rows_of_large_tiles(ep, cap):
    H = F = 1032
    counts = block_case(cap, H, F)
    g, n, off = gen(21), sum(counts), offsets_of(counts)
    x, up, down = plain.block_inputs(g, counts, H, F, torch.bfloat16)
    gate_up, act, dy = (plain.randn(g, n, k, dtype=torch.bfloat16) for k in (2 * F, F, H))

    def both(f):
        outs = [f(torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")) for k in (F, H, 2 * F, 2 * F, H)]
        grads = [torch.empty_like(up), torch.empty_like(down)]
        ep.ep_expert_ffn(f(x), up, down, outs[0], outs[1], gate_up=outs[2], expert_offsets=off)
        ep.ep_expert_ffn_backward(f(dy), f(x), f(gate_up), f(act), up, down, outs[3], outs[4], *grads, expert_offsets=off)
        return outs + grads

    for a, b in zip(both(lambda t: t), both(lambda t: plain.strided(t, 24))):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ rows of nobody

ALIGNED = [([0, 128, 128, 256], [100, 0, 3]), ([0, 40, 80, 120], [40, 0, 17]), ([0, 300, 600, 900], [1, 300, 129]),
           ([128 * k for k in range(49)], [1 + 53 * k % 128 for k in range(48)])]


def layout(offsets, counts):
    rows = offsets[-1]
    real = torch.tensor([r - offsets[e] < counts[e] for e in range(len(counts)) for r in range(offsets[e], offsets[e + 1])]).cuda()
    off, cnt = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (offsets, counts))
    return rows, real, off, cnt


@pytest.mark.parametrize("offsets,counts", ALIGNED)
def test_gradients_of_aligned_and_strided_layouts(ep, offsets, counts):
    """Rows behind an expert's last are NaN in every input: they enter nothing and none of theirs is written. The same bits as with
    the real rows one expert after the other, for what does not depend on how tiles are cut: the weights' gradients."""
    H, F, E = 136, 72, len(counts)
    rows, real, off, cnt = layout(offsets, counts)
    g = gen(rows)
    x, up, down = plain.block_inputs(g, [rows] + [0] * (E - 1), H, F, torch.bfloat16)
    gate_up, act, dy = (plain.randn(g, rows, k, dtype=torch.bfloat16) for k in (2 * F, F, H))
    for t in (x, gate_up, act, dy):
        t[~real] = math.nan
    outs = [torch.full((rows, k), 7.0, dtype=torch.bfloat16, device="cuda") for k in (2 * F, H)]
    grads = [torch.full_like(t, math.nan) for t in (up, down)]
    ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, *outs, *grads, expert_offsets=off, expert_counts=cnt)
    dense = [torch.empty(sum(counts), k, dtype=torch.bfloat16, device="cuda") for k in (2 * F, H)]
    dense_grads = [torch.empty_like(t) for t in (up, down)]
    ep.ep_expert_ffn_backward(*(t[real] for t in (dy, x, gate_up, act)), up, down, *dense, *dense_grads, expert_offsets=offsets_of(counts))
    for a, b in zip(outs + grads, dense + dense_grads):
        got = a if a.dim() == 3 else a[real]
        assert torch.equal(got, b)
        assert a.dim() == 3 or (a[~real] == 7).all()


@pytest.mark.parametrize("offsets,counts", ALIGNED)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("quantised", [False, True])
def test_fp8_rows_of_aligned_and_strided_layouts(ep, offsets, counts, swiglu, quantised):
    rows, real, off, cnt = layout(offsets, counts)
    g, cols = gen(rows), 640
    x, xs = fp8_rows(g, rows, 256)
    w, ws = fp8_weights(g, len(counts), 2 * cols if swiglu else cols, 256)
    xs[~real] = math.nan
    y = torch.full((rows, cols), 7.0, device="cuda").to(E4M3 if quantised else torch.bfloat16)
    ys = torch.full((rows, cols // 128), 7.0, device="cuda") if quantised else None
    ep.ep_expert_fp8(x, xs, w, ws, y, expert_offsets=off, expert_counts=cnt, y_scales=ys, activation=int(swiglu))
    want, tol = fp8_reference(counts, x[real], xs[real], w, ws, swiglu)
    assert (y[~real].float() == 7).all()
    if not quantised:
        return within(y[real], want, tol + U[y.dtype] * want.abs())
    assert (ys[~real] == 7).all()
    wide = ys[real].double().repeat_interleave(128, 1)
    within(y[real].double() * wide, want, tol + (want.abs() + tol) * 2.0 ** -4 + 2.0 ** -10 * wide)


@pytest.mark.parametrize("rows", [1, 40, 300, 5000])
def test_one_expert_without_offsets(ep, rows):
    H, F, g = 264, 136, gen(rows)
    x, up, down = plain.block_inputs(g, [rows], H, F, torch.float16)
    dy = plain.randn(g, rows, H, dtype=torch.float16)

    def step(**kw):
        act, y, gate_up, dgu, dx = (torch.empty(rows, k, dtype=torch.float16, device="cuda") for k in (F, H, 2 * F, 2 * F, H))
        grads = [torch.empty_like(up), torch.empty_like(down)]
        ep.ep_expert_ffn(x, up, down, act, y, gate_up=gate_up, **kw)
        ep.ep_expert_ffn_backward(dy, x, gate_up, act, up, down, dgu, dx, *grads, **kw)
        return act, y, gate_up, dgu, dx, *grads

    for a, b in zip(step(), step(expert_offsets=offsets_of([rows]))):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ streams and graphs

def mixed_calls(ep):
    """Calls of all forms on buffers of their own: (call(stream), its outputs)."""
    calls = []
    for counts, I, O in (([3], 2048, 512), (FP8_COUNTS["lanes"], 256, 768), (FP8_COUNTS[64], 384, 640)):
        g, n = gen(I), sum(counts)
        x, xs = fp8_rows(g, n, I)
        w, ws = fp8_weights(g, len(counts), O, I)
        y, off = torch.empty(n, O, dtype=torch.bfloat16, device="cuda"), offsets_of(counts)
        calls.append((lambda s, a=(x, xs, w, ws, y), o=off: ep.ep_expert_fp8(*a, expert_offsets=o, stream=s), [y]))
    for cap in (64, 256):
        counts, H, F = BLOCK_COUNTS[cap], 520, 264
        g, n, off = gen(cap), sum(counts), offsets_of(counts)
        x, up, down = plain.block_inputs(g, counts, H, F, torch.bfloat16)
        outs = [torch.empty(n, k, dtype=torch.bfloat16, device="cuda") for k in (F, H, 2 * F, 2 * F, H)] + [torch.empty_like(up), torch.empty_like(down)]

        def step(s, a=(x, up, down), outs=outs, off=off):
            ep.ep_expert_ffn(*a, outs[0], outs[1], gate_up=outs[2], expert_offsets=off, stream=s)
            ep.ep_expert_ffn_backward(a[0], a[0], outs[2], outs[0], a[1], a[2], *outs[3:], expert_offsets=off, stream=s)

        calls.append((step, outs))
    return calls


def test_all_forms_at_once_on_streams_of_their_own(ep):
    calls = mixed_calls(ep)
    for call, _ in calls:
        call(None)
    want = [[t.clone() for t in outs] for _, outs in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, (call, _) in zip(streams, calls):
            call(s)
    torch.cuda.synchronize()
    for (_, outs), w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))


def test_all_forms_in_two_graphs_at_once(ep):
    """Two graphs of all forms, each captured on a stream of its own and replayed beside the other."""
    sets = [mixed_calls(ep) for _ in range(2)]
    for call, _ in sets[0]:
        call(None)
    want = [t.clone() for _, outs in sets[0] for t in outs]
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in sets], []
    for s, calls in zip(streams, sets):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for call, _ in calls:
                call(None)
        graphs.append(graph)
    for calls in sets:
        for _, outs in calls:
            for t in outs:
                t.fill_(math.nan)
    torch.cuda.synchronize()
    for _ in range(10):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for calls in sets:
        assert all(torch.equal(a, b) for a, b in zip([t for _, outs in calls for t in outs], want))
