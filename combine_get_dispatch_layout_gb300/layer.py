"""Binding of the layer operators (include/ep_layer.h): router top-k and its
gradient, append to a paged cache, attention of one new token over it, and the
experts' products: with 4-bit weights, in 8-bit floating point, and the gated
block in 16 bits with its gradients.

As in the package itself, each function has the name of the C entry point and
only marshals arguments; sizes, strides and types come from the tensors. What
the C ABI cannot see (a tensor's type, its device, the memory its strides
reach) raises ValueError before the call. The marshalling is compiled
(csrc/layer_bind.cpp): a decode step makes these calls for a few microseconds of
GPU work each. Like libep.so it is built by build.py, and without it the first
call raises.
"""
from __future__ import annotations

import ctypes
import importlib

import torch

from . import EP_DTYPE_BF16, EP_DTYPE_FP16, EP_ERR_INVALID_ARG, EP_OK, EP_SCALE_FP32, _LIB_PATH, EPError, lib

EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
EP_ACT_NONE, EP_ACT_SWIGLU = 0, 1

EXPORTS = ("ep_router_topk", "ep_router_topk_backward", "ep_kv_append", "ep_paged_attention",
           "ep_paged_attention_workspace", "ep_expert_w4", "ep_expert_w4_workspace", "ep_expert_fp8", "ep_expert_ffn",
           "ep_expert_ffn_backward")

_i32, _i64, _f32, _P = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


# The C ABI's structures and argument types, for callers through ctypes (and for the check that they match the header);
# the functions below go through the compiled marshalling.

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


class Fp8Config(ctypes.Structure):
    """ep_fp8_config_t (include/ep_layer.h)."""
    _fields_ = [("x_dtype", _i32), ("y_dtype", _i32), ("activation", _i32), ("x_scale_mode", _i32),
                ("y_scale_mode", _i32), ("x_ld", _i64), ("y_ld", _i64), ("x_scale_row", _i64), ("x_scale_block", _i64),
                ("y_scale_row", _i64), ("y_scale_block", _i64)]


class FfnConfig(ctypes.Structure):
    """ep_ffn_config_t (include/ep_layer.h)."""
    _fields_ = [("dtype", _i32), ("grad_w_dtype", _i32), ("accumulate", _i32), ("x_ld", _i64), ("gate_up_ld", _i64),
                ("act_ld", _i64), ("y_ld", _i64), ("grad_x_ld", _i64), ("grad_gate_up_ld", _i64)]


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
    L.ep_expert_fp8.argtypes = [_P, _P, _i64, _i32, _P, _P, _P, _P, _i32, _i32, ref(Fp8Config), _P, _P, _P]
    L.ep_expert_ffn.argtypes = [_P, _i64, _i32, _P, _P, _P, _P, _i32, _i32, ref(FfnConfig), _P, _P, _P, _P]
    L.ep_expert_ffn_backward.argtypes = [_P, _P, _P, _P, _i64, _i32, _P, _P, _P, _P, _i32, _i32, ref(FfnConfig), _P, _P,
                                         _P, _P, _P]
    for name in EXPORTS:
        getattr(L, name).restype = _i64 if name.endswith("workspace") else _i32


_bound = None


def _bind():
    """The compiled marshalling, opened on the library (raises if either has not been built)."""
    global _bound
    if _bound is None:
        lib()
        try:
            module = importlib.import_module("._layer_bind", __package__)
        except ImportError as e:
            raise RuntimeError(f"the layer binding is not built for this torch ({e}); run {__package__}.build.build()") from e
        module.open(_LIB_PATH)
        _bound = module
    return _bound


def _check(st: int, call: str) -> None:
    if st != EP_OK:
        raise EPError(st, call)


def ep_router_topk(logits, topk_idx, topk_weights, bias=None, score: int = EP_SCORE_SOFTMAX, renormalize: bool = True,
                   scale: float = 1.0, num_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
                   stream=None) -> None:
    """topk_idx [T, K] int64 and topk_weights [T, K] fp32 from logits [T, E]."""
    _check((_bound or _bind()).router_topk(logits, topk_idx, topk_weights, bias, score, renormalize, scale, num_groups,
                                           topk_groups, group_top, stream), "ep_router_topk")


def ep_router_topk_backward(logits, topk_idx, grad_weights, grad_logits, score: int = EP_SCORE_SOFTMAX,
                            renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """grad_logits [T, E] (the logits' type) from grad_weights [T, K] fp32 at the experts topk_idx."""
    _check((_bound or _bind()).router_topk_backward(logits, topk_idx, grad_weights, grad_logits, score, renormalize,
                                                    scale, stream), "ep_router_topk_backward")


def ep_kv_append(q, k, v, positions, slots, cos_sin, q_out, k_cache, v_cache, interleaved: bool = False,
                 k_scale: float = 1.0, v_scale: float = 1.0, device_error=None, stream=None) -> None:
    """Turn q [T, heads, D] into q_out and k [T, kv_heads, D] on its way to the
    cache [pages, page_size, kv_heads, D], v unturned, at slots [T] int64 (-1:
    not cached). cos_sin [max_position, rotary_dim] fp32, or None for no
    rotation; q and q_out may be None. The cache's first three dimensions may lie
    in any order in memory."""
    _check((_bound or _bind()).kv_append(q, k, v, positions, slots, cos_sin, q_out, k_cache, v_cache, interleaved,
                                         k_scale, v_scale, device_error, stream), "ep_kv_append")


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
    _check((_bound or _bind()).paged_attention(q, k_cache, v_cache, block_table, seq_lens, out, workspace, lse, scale,
                                               window, k_scale, v_scale, stream), "ep_paged_attention")


def ep_expert_w4(x, weights, scales, y, expert_offsets=None, expert_counts=None, zeros=None,
                 activation: int = EP_ACT_NONE, workspace=None, stream=None) -> None:
    """y [rows, O] (O/2 columns with EP_ACT_SWIGLU) = x [rows, I] times each
    row's expert's weights [E, O, I/2] uint8, two 4-bit codes a byte, with
    scales [E, I/group, O] of x's type and zeros [E, I/group, O] uint8 (8
    if None). Rows belong to experts by expert_offsets [E + 1] int32 (None: one
    expert); with expert_counts [E] int32 only each expert's first rows count.
    Without a workspace (ep_expert_w4_workspace bytes) one is taken from torch's
    allocator for the call, on the current stream only."""
    _check((_bound or _bind()).expert_w4(x, weights, scales, y, expert_offsets, expert_counts, zeros, activation,
                                         workspace, stream), "ep_expert_w4")


def ep_expert_w4_workspace(x, scales) -> int:
    """Bytes of workspace that ep_expert_w4 needs for tensors of these shapes."""
    rows, I = x.shape
    kind = {torch.bfloat16: EP_DTYPE_BF16, torch.float16: EP_DTYPE_FP16}.get(x.dtype, -1)
    size = lib().ep_expert_w4_workspace(rows, I, I // max(scales.shape[1], 1), kind)
    if size < 0:
        raise EPError(EP_ERR_INVALID_ARG, "ep_expert_w4_workspace")
    return size


def ep_expert_fp8(x, x_scales, weights, weight_scales, y, expert_offsets=None, expert_counts=None,
                  activation: int = EP_ACT_NONE, y_scales=None, scale_mode: int = EP_SCALE_FP32, stream=None) -> None:
    """y [rows, O] (O/2 columns with EP_ACT_SWIGLU) = x [rows, I] (float8_e4m3fn
    or float8_e5m2, the fp8 dispatch's bytes by .view()) with x_scales
    [rows, I/128] (fp32, or uint8 exponents; a transposed view for column-major
    scales) times each row's expert's weights [E, O, I] float8_e4m3fn with
    weight_scales [E, ceil(O/128), I/128] fp32. y is bf16 or fp16, or
    float8_e4m3fn with y_scales [rows, columns/128] (fp32 by scale_mode, or uint8
    exponents), which the next call takes as x and x_scales. Rows belong to
    experts by expert_offsets [E + 1] int32 (None: one expert); with
    expert_counts [E] int32 only each expert's first rows count."""
    _check((_bound or _bind()).expert_fp8(x, x_scales, weights, weight_scales, y, y_scales, expert_offsets, expert_counts,
                                          activation, scale_mode, stream), "ep_expert_fp8")


def ep_expert_ffn(x, w_gate_up, w_down, act, y, gate_up=None, expert_offsets=None, expert_counts=None,
                  stream=None) -> None:
    """act [rows, F] = silu(gate) * up with (gate, up) = w_gate_up [E, 2F, H] x
    [rows, H], and y [rows, H] = w_down [E, H, F] act, by expert as in
    ep_expert_fp8, all bf16 or all fp16. gate_up [rows, 2F], if given, gets gate
    and up for the backward call. w_down and y may be None: act alone."""
    _check((_bound or _bind()).expert_ffn(x, w_gate_up, w_down, act, y, gate_up, expert_offsets, expert_counts, stream),
           "ep_expert_ffn")


def ep_expert_ffn_backward(grad_y, x, gate_up, act, w_gate_up, w_down, grad_gate_up, grad_x=None, grad_w_gate_up=None,
                           grad_w_down=None, expert_offsets=None, expert_counts=None, accumulate: bool = False,
                           stream=None) -> None:
    """Gradients of ep_expert_ffn from grad_y [rows, H]: grad_gate_up [rows, 2F]
    and those of grad_x [rows, H], grad_w_gate_up [E, 2F, H] and grad_w_down
    [E, H, F] that are given. The weights' are of the tensors' type or fp32, and
    with accumulate they are added to what is there. x is needed for
    grad_w_gate_up only, act for grad_w_down and w_gate_up for grad_x.
    grad_gate_up may be gate_up itself, grad_x may be grad_y."""
    _check((_bound or _bind()).expert_ffn_backward(grad_y, x, gate_up, act, w_gate_up, w_down, grad_gate_up, grad_x,
                                                   grad_w_gate_up, grad_w_down, expert_offsets, expert_counts, accumulate,
                                                   stream), "ep_expert_ffn_backward")
