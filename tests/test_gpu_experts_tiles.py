"""The experts' products at sizes that take the larger tiles: every shape of the kernels, beside one another in a call."""
import math

import pytest
import torch

from test_gpu_experts import F32, TINY, U, ep, fp8_reference, fp8_rows, fp8_weights, gen, offsets_of, within  # noqa: F401

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
