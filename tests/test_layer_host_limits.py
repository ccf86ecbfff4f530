"""CPU-only checks of the layer operators' C ABI at the ends of what it takes
(the addresses here are never dereferenced)."""
import pytest

from test_layer_host import INVALID, append, cache_struct, ep, experts  # noqa: F401  (ep: fixture)


@pytest.mark.parametrize("kw", [dict(k_scale=1e-39), dict(v_scale=2.0 ** -128)])
def test_append_rejects_scales_without_a_reciprocal(ep, kw):
    """1 / scale is infinite in fp32: a zero would be stored as NaN."""
    cache = cache_struct(ep, dtype=ep.EP_DTYPE_FP8_E4M3, **kw)
    assert append(ep, cache) == INVALID


@pytest.mark.parametrize("kw", [dict(O=2 ** 31 - 511, y_ld=2 ** 31), dict(O=2 ** 31 - 2, y_ld=2 ** 31, act=1),
                                dict(I=2 ** 31 - 64, x_ld=2 ** 31), dict(rows=2 ** 31 - 1)])
def test_experts_reject_sizes_whose_tiles_pass_an_int(ep, kw):
    assert experts(ep, **{"rows": 9, **kw}) == INVALID


def test_experts_workspace_rejects_sizes_whose_tiles_pass_an_int(ep):
    assert ep.lib().ep_expert_w4_workspace(2 ** 31 - 1, 64, 64, 0) == -1
    assert ep.lib().ep_expert_w4_workspace(9, 2 ** 31 - 64, 64, 0) == -1
    assert ep.lib().ep_expert_w4_workspace(9, 2 ** 31 - 512, 64, 0) > 0
