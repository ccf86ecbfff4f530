"""Binding of the layer operators (include/ep_layer.h): router top-k and its
gradient, append to a paged cache, attention of one new token over it, and the
experts' products with 4-bit weights.

As in the package itself, each function has the name of the C entry point and
only marshals arguments; sizes, strides and types come from the tensors. What
the C ABI cannot see (a tensor's type, its device, the memory its strides
reach) is checked here and raises ValueError before the call.
"""
from __future__ import annotations

import ctypes

import torch

from . import (EP_DTYPE_BF16, EP_DTYPE_FP8_E4M3, EP_DTYPE_FP16, EP_DTYPE_FP32, EP_ERR_INVALID_ARG, EPError, _check,
               _stream, lib)

EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
EP_ACT_NONE, EP_ACT_SWIGLU = 0, 1

EXPORTS = ("ep_router_topk", "ep_router_topk_backward", "ep_kv_append", "ep_paged_attention",
           "ep_paged_attention_workspace", "ep_expert_w4", "ep_expert_w4_workspace")

_i32, _i64, _f32, _P = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class RouterConfig(ctypes.Structure):
    """ep_router_config_t (include/ep_layer.h)."""
    _fields_ = [("logits_dtype", _i32), ("score", _i32), ("renormalize", _i32), ("scale", _f32),
                ("num_groups", _i32), ("topk_groups", _i32), ("group_top", _i32)]


class Cache(ctypes.Structure):
    """ep_cache_t (include/ep_layer.h)."""
    _fields_ = [("dtype", _i32), ("page_size", _i32), ("num_pages", _i64), ("k_page_stride", _i64),
                ("k_slot_stride", _i64), ("k_head_stride", _i64), ("v_page_stride", _i64), ("v_slot_stride", _i64),
                ("v_head_stride", _i64), ("k_scale", _f32), ("v_scale", _f32)]


class AppendConfig(ctypes.Structure):
    """ep_append_config_t (include/ep_layer.h)."""
    _fields_ = [("dtype", _i32), ("num_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32),
                ("rotary_dim", _i32), ("interleaved", _i32), ("q_ld", _i64), ("k_ld", _i64), ("v_ld", _i64),
                ("q_out_ld", _i64), ("max_position", _i64)]


class AttentionConfig(ctypes.Structure):
    """ep_attention_config_t (include/ep_layer.h)."""
    _fields_ = [("dtype", _i32), ("num_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("max_pages", _i32),
                ("q_ld", _i64), ("out_ld", _i64), ("table_ld", _i64), ("scale", _f32), ("window", _i32)]


class W4Config(ctypes.Structure):
    """ep_w4_config_t (include/ep_layer.h)."""
    _fields_ = [("dtype", _i32), ("group_size", _i32), ("activation", _i32), ("x_ld", _i64), ("y_ld", _i64)]


def declare(L) -> None:
    """Argument types of this module's entry points on a loaded library."""
    ref = ctypes.POINTER
    L.ep_router_topk.argtypes = [_P, _i64, _P, _i32, _i32, _i32, ref(RouterConfig), _P, _P, _P]
    L.ep_router_topk_backward.argtypes = [_P, _i64, _P, _i64, _P, _i32, _i32, _i32, ref(RouterConfig), _P, _i64, _P]
    L.ep_kv_append.argtypes = [_P, _P, _P, _P, _P, _P, _i32, ref(AppendConfig), _P, _P, _P, ref(Cache), _P, _P]
    L.ep_paged_attention.argtypes = [_P, _P, _P, ref(Cache), _P, _P, _i32, ref(AttentionConfig), _P, _P, _P, _i64, _P]
    L.ep_paged_attention_workspace.argtypes = [_i32, _i32, _i32, _i32]
    L.ep_expert_w4.argtypes = [_P, _i64, _i32, _P, _P, _P, _P, _P, _i32, _i32, ref(W4Config), _P, _P, _i64, _P]
    L.ep_expert_w4_workspace.argtypes = [_i64, _i32, _i32, _i32]
    for name in EXPORTS:
        getattr(L, name).restype = _i64 if name.endswith("workspace") else _i32


_FLOATS = {torch.bfloat16: EP_DTYPE_BF16, torch.float16: EP_DTYPE_FP16}
_LOGITS = {**_FLOATS, torch.float32: EP_DTYPE_FP32}
_CACHES = {**_FLOATS, torch.float8_e4m3fn: EP_DTYPE_FP8_E4M3}


def _dtype(t, known, what: str) -> int:
    d = known.get(t.dtype)
    if d is None:
        raise ValueError(f"{what}: {t.dtype} is not supported")
    return d


# A decode step makes these calls for a few microseconds of GPU work each, so the checks are kept to a few
# attribute reads a tensor, and the current stream is read without building a Stream object (2.8 us).
def _raw_stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return _stream(stream)


def _on_gpu(t, what: str) -> int:
    """Address of a tensor whose strides the call is given."""
    if not t.is_cuda and t.numel() > 0 and not t.is_pinned():
        raise ValueError(f"{what} must be a CUDA tensor or a pinned host tensor")
    return t.data_ptr()


def _dense(t, dtype, shape, what: str):
    """Address of a contiguous tensor of this type and shape (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr() if t.is_cuda else _on_gpu(t, what)


def _rows(t, dtype, shape, what: str) -> tuple[int, int]:
    """(address, elements from row to row) of a tensor whose rows are dense."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    strides = t.stride()
    step = 1
    for k in range(len(shape) - 1, 0, -1):
        if strides[k] != step and shape[k] != 1:
            raise ValueError(f"{what}: all but the first dimension must be contiguous")
        step *= shape[k]
    return t.data_ptr() if t.is_cuda else _on_gpu(t, what), strides[0] if shape[0] > 1 else -(-step // 8) * 8


def ep_router_topk(logits, topk_idx, topk_weights, bias=None, score: int = EP_SCORE_SOFTMAX, renormalize: bool = True,
                   scale: float = 1.0, num_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
                   stream=None) -> None:
    """topk_idx [T, K] int64 and topk_weights [T, K] fp32 from logits [T, E]."""
    T, E = logits.shape
    K = topk_idx.shape[1]
    cfg = RouterConfig(_dtype(logits, _LOGITS, "logits"), score, bool(renormalize), scale, num_groups, topk_groups,
                       group_top)
    p, ld = _rows(logits, logits.dtype, (T, E), "logits")
    _check(lib().ep_router_topk(p, ld, _dense(bias, torch.float32, (E,), "bias"), T, E, K, cfg,
                                _dense(topk_idx, torch.int64, (T, K), "topk_idx"),
                                _dense(topk_weights, torch.float32, (T, K), "topk_weights"), _raw_stream(stream)),
           "ep_router_topk")


def ep_router_topk_backward(logits, topk_idx, grad_weights, grad_logits, score: int = EP_SCORE_SOFTMAX,
                            renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """grad_logits [T, E] (the logits' type) from grad_weights [T, K] fp32 at the experts topk_idx."""
    T, E = logits.shape
    K = topk_idx.shape[1]
    cfg = RouterConfig(_dtype(logits, _LOGITS, "logits"), score, bool(renormalize), scale, 1, 1, 1)
    p, ld = _rows(logits, logits.dtype, (T, E), "logits")
    gp, gld = _rows(grad_logits, logits.dtype, (T, E), "grad_logits")
    ip, ild = _rows(topk_idx, torch.int64, (T, K), "topk_idx")
    _check(lib().ep_router_topk_backward(p, ld, ip, ild,
                                         _dense(grad_weights, torch.float32, (T, K), "grad_weights"), T, E, K, cfg,
                                         gp, gld, _raw_stream(stream)),
           "ep_router_topk_backward")


def _cache(k_cache, v_cache, k_scale: float, v_scale: float, heads: int, dim: int) -> Cache:
    """ep_cache_t of two [pages, page_size, heads, dim] tensors, in any order of the first three in memory."""
    shape = k_cache.shape
    if shape != v_cache.shape or k_cache.dtype is not v_cache.dtype or len(shape) != 4:
        raise ValueError("k_cache and v_cache must be [pages, page_size, kv_heads, head_dim] of one type")
    pages, page, h, d = shape
    if h != heads or d != dim:
        raise ValueError(f"cache rows are [{h}, {d}], the call's are [{heads}, {dim}]")
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("the cache's last dimension must be contiguous")
    return Cache(_dtype(k_cache, _CACHES, "cache"), page, pages, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], k_scale,
                 v_scale)


def ep_kv_append(q, k, v, positions, slots, cos_sin, q_out, k_cache, v_cache, interleaved: bool = False,
                 k_scale: float = 1.0, v_scale: float = 1.0, device_error=None, stream=None) -> None:
    """Turn q [T, heads, D] into q_out and k [T, kv_heads, D] on its way to the
    cache [pages, page_size, kv_heads, D], v unturned, at slots [T] int64 (-1:
    not cached). cos_sin [max_position, rotary_dim] fp32, or None for no
    rotation; q and q_out may be None."""
    T, n, d = k.shape
    dt = _dtype(k, _FLOATS, "k")
    kp, kld = _rows(k, k.dtype, (T, n, d), "k")
    vp, vld = _rows(v, k.dtype, (T, n, d), "v")
    qp = qop = None
    h = qld = qold = 0
    if q is not None:
        h = q.shape[1]
        qp, qld = _rows(q, k.dtype, (T, h, d), "q")
        qop, qold = _rows(q_out, k.dtype, (T, h, d), "q_out")
    most, rot = cos_sin.shape if cos_sin is not None else (0, 0)
    cache = _cache(k_cache, v_cache, k_scale, v_scale, n, d)
    cfg = AppendConfig(dt, h, n, d, rot, bool(interleaved), qld, kld, vld, qold, most)
    _check(lib().ep_kv_append(qp, kp, vp, _dense(positions, torch.int64, (T,), "positions"),
                              _dense(slots, torch.int64, (T,), "slots"),
                              _dense(cos_sin, torch.float32, (most, rot), "cos_sin"), T, cfg, qop,
                              _on_gpu(k_cache, "k_cache"), _on_gpu(v_cache, "v_cache"), cache,
                              _dense(device_error, torch.int32, (1,), "device_error"), _raw_stream(stream)),
           "ep_kv_append")


def ep_paged_attention_workspace(q, k_cache, block_table) -> int:
    """Bytes of workspace that ep_paged_attention needs for tensors of these shapes."""
    B, h, d = q.shape
    size = lib().ep_paged_attention_workspace(B, h, k_cache.shape[2], d)
    if size < 0:
        raise ValueError(f"no attention of {h} heads over {k_cache.shape[2]}, head_dim {d}")
    return size


def ep_paged_attention(q, k_cache, v_cache, block_table, seq_lens, out, workspace, lse=None,
                       scale: float | None = None, window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0,
                       stream=None) -> None:
    """out [B, heads, D] = attention of q [B, heads, D] over each sequence's
    first seq_lens[b] keys in the cache [pages, page_size, kv_heads, D], page by
    page through block_table [B, max_pages] int32. scale defaults to
    1 / sqrt(D)."""
    B, h, d = q.shape
    n = k_cache.shape[2]
    dt = _dtype(q, _FLOATS, "q")
    qp, qld = _rows(q, q.dtype, (B, h, d), "q")
    op, old = _rows(out, q.dtype, (B, h, d), "out")
    pages = block_table.shape[1]
    tp, tld = _rows(block_table, torch.int32, (B, pages), "block_table")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, n, d)
    cfg = AttentionConfig(dt, h, n, d, pages, qld, old, tld, d ** -0.5 if scale is None else scale, window)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check(lib().ep_paged_attention(qp, _on_gpu(k_cache, "k_cache"), _on_gpu(v_cache, "v_cache"), cache, tp,
                                    _dense(seq_lens, torch.int32, (B,), "seq_lens"), B, cfg, op,
                                    _dense(lse, torch.float32, (B, h), "lse"), _on_gpu(workspace, "workspace"),
                                    workspace.numel() * workspace.element_size(), _raw_stream(stream)),
           "ep_paged_attention")


def ep_expert_w4(x, weights, scales, y, expert_offsets=None, expert_counts=None, zeros=None,
                 activation: int = EP_ACT_NONE, workspace=None, stream=None) -> None:
    """y [rows, O] (O/2 columns with EP_ACT_SWIGLU) = x [rows, I] times each
    row's expert's weights [E, O, I/2] uint8, two 4-bit codes a byte, with
    scales [E, I/group, O] of x's type and zeros [E, I/group, O] uint8 (8
    if None). Rows belong to experts by expert_offsets [E + 1] int32 (None: one
    expert); with expert_counts [E] int32 only each expert's first rows count.
    Without a workspace (ep_expert_w4_workspace bytes) one is taken from torch's
    allocator for the call, on the current stream only."""
    rows, I = x.shape
    E, O, half = weights.shape
    groups = scales.shape[1]
    if 2 * half != I or groups < 1 or I % groups != 0:
        raise ValueError(f"weights [{E}, {O}, {half}] and {groups} groups do not fit rows of {I}")
    xp, xld = _rows(x, x.dtype, (rows, I), "x")
    yp, yld = _rows(y, x.dtype, (rows, O // 2 if activation == EP_ACT_SWIGLU else O), "y")
    cfg = W4Config(_dtype(x, _FLOATS, "x"), I // groups, activation, xld, yld)
    if workspace is None:
        if stream is not None:
            raise ValueError("a call on a stream of its own needs a workspace")
        workspace = torch.empty(max(ep_expert_w4_workspace(x, scales), 0), dtype=torch.uint8, device=x.device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check(lib().ep_expert_w4(xp, rows, I, _dense(weights, torch.uint8, (E, O, half), "weights"),
                              _dense(scales, x.dtype, (E, groups, O), "scales"),
                              _dense(zeros, torch.uint8, (E, groups, O), "zeros"),
                              _dense(expert_offsets, torch.int32, (E + 1,), "expert_offsets"),
                              _dense(expert_counts, torch.int32, (E,), "expert_counts"), E, O, cfg, yp,
                              _on_gpu(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                              _raw_stream(stream)),
           "ep_expert_w4")


def ep_expert_w4_workspace(x, scales) -> int:
    """Bytes of workspace that ep_expert_w4 needs for tensors of these shapes."""
    rows, I = x.shape
    size = lib().ep_expert_w4_workspace(rows, I, I // max(scales.shape[1], 1), _dtype(x, _FLOATS, "x"))
    if size < 0:
        raise EPError(EP_ERR_INVALID_ARG, "ep_expert_w4_workspace")
    return size
