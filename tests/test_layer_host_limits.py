"""CPU-only checks of the layer operators' C ABI at the ends of what it takes
(the addresses here are never dereferenced)."""
import pytest

from test_layer_host import INVALID, append, cache_struct, ep, experts  # noqa: F401  (ep: fixture)


@pytest.mark.parametrize("kw", [dict(k_scale=1e-39), dict(v_scale=2.0 ** -128)])
def test_append_rejects_scales_without_a_reciprocal(ep, kw):
    """1 / scale is infinite in fp32: a zero would be stored as NaN."""
    cache = cache_struct(ep, dtype=ep.EP_DTYPE_FP8_E4M3, **kw)
    assert append(ep, cache) == INVALID
