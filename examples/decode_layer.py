"""One decode step of a transformer layer with experts, every heavy part through the library.

    python examples/decode_layer.py [--tokens 64] [--steps 20]

A step takes one new token of each of T sequences through

  4-bit projection to queries, keys, values   ep_expert_w4 (one matrix)
  rotation and append to the paged cache      ep_kv_append
  attention over the cache                    ep_paged_attention
  4-bit output projection                     ep_expert_w4
  router                                      ep_router_topk (logits: a plain matrix product)
  layout, dispatch                            ep_layout, ep_dispatch_ex
  experts, gate and up with the activation    ep_expert_w4 (the layout's offsets)
  experts, down                               ep_expert_w4
  weighted combine                            ep_combine

with the norms and residual sums between them as plain torch operations. Buffers are made once, the step enqueues work
only, and main() captures it into a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_get_dispatch_layout_gb300 as ep  # noqa: E402


def quantised(experts: int, rows: int, inputs: int, group: int, generator):
    """Random 4-bit weights [experts, rows, inputs/2] with scales that keep outputs near their inputs' size."""
    codes = torch.randint(0, 256, (experts, rows, inputs // 2), dtype=torch.uint8, device="cuda", generator=generator)
    scales = torch.rand(experts, inputs // group, rows, device="cuda", generator=generator) + 0.5
    return codes, (scales / (4.6 * inputs ** 0.5)).bfloat16()


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(1, keepdim=True) + 1e-6)).bfloat16()


class DecodeLayer:
    """Weights, cache and buffers of one layer for T sequences of at most max_len tokens."""

    def __init__(self, T: int, hidden: int = 2048, heads: int = 16, kv_heads: int = 4, dim: int = 128, experts: int = 64,
                 topk: int = 6, inner: int = 1024, page: int = 64, max_len: int = 4096, group: int = 128, seed: int = 0):
        g = torch.Generator("cuda").manual_seed(seed)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.T, self.heads, self.kv_heads, self.dim, self.experts, self.topk = T, heads, kv_heads, dim, experts, topk
        self.page = page
        rows = (heads + 2 * kv_heads) * dim
        self.w_qkv, self.s_qkv = quantised(1, rows, hidden, group, g)
        self.w_out, self.s_out = quantised(1, hidden, heads * dim, group, g)
        self.w_up, self.s_up = quantised(experts, 2 * inner, hidden, group, g)
        self.w_down, self.s_down = quantised(experts, hidden, inner, group, g)
        self.gate = (torch.randn(experts, hidden, device="cuda", generator=g) / hidden ** 0.5).bfloat16()
        # the cache: every sequence owns max_len / page pages, scattered
        per_seq = -(-max_len // page)
        order = torch.randperm(T * per_seq, device="cuda", generator=g)
        self.block_table = order.to(torch.int32).view(T, per_seq)
        self.k_cache = torch.zeros(T * per_seq, page, kv_heads, dim, **bf16)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.seq_lens = torch.zeros(T, dtype=torch.int32, device="cuda")
        angle = torch.arange(max_len, device="cuda")[:, None] * 10000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1)
        # buffers
        self.qkv = torch.empty(T, rows, **bf16)
        self.q = torch.empty(T, heads, dim, **bf16)
        self.attended = torch.empty(T, heads, dim, **bf16)
        self.projected = torch.empty(T, hidden, **bf16)
        self.idx = torch.empty(T, topk, dtype=torch.int64, device="cuda")
        self.weights = torch.empty(T, topk, device="cuda")
        self.counts = torch.empty(experts, dtype=torch.int32, device="cuda")
        self.rank_tokens = torch.empty(1, dtype=torch.int32, device="cuda")
        self.in_rank = torch.empty(T, 1, dtype=torch.uint8, device="cuda")
        self.offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
        self.received = torch.empty(T * topk, hidden, **bf16)
        self.activated = torch.empty(T * topk, inner, **bf16)
        self.returned = torch.empty(T * topk, hidden, **bf16)
        self.combined = torch.empty(T, hidden, **bf16)
        self.handle = None
        work = ep.ep_paged_attention_workspace(self.q, self.k_cache, self.block_table)
        self.attention_work = torch.empty(work, dtype=torch.uint8, device="cuda")

    def attention(self, x):
        """x plus the attention of its new tokens, which join the cache."""
        positions = self.seq_lens.long()
        page = self.block_table.gather(1, (positions // self.page)[:, None])[:, 0].long()
        ep.ep_expert_w4(norm(x), self.w_qkv, self.s_qkv, self.qkv)
        q, k, v = self.qkv.unflatten(1, (-1, self.dim)).split((self.heads, self.kv_heads, self.kv_heads), 1)
        ep.ep_kv_append(q, k, v, positions, page * self.page + positions % self.page, self.cos_sin, self.q, self.k_cache,
                        self.v_cache)
        self.seq_lens += 1
        ep.ep_paged_attention(self.q, self.k_cache, self.v_cache, self.block_table, self.seq_lens, self.attended,
                              self.attention_work)
        ep.ep_expert_w4(self.attended.flatten(1), self.w_out, self.s_out, self.projected)
        return x + self.projected

    def mixture(self, x):
        """x plus its experts' outputs."""
        h = norm(x)
        ep.ep_router_topk(h @ self.gate.t(), self.idx, self.weights)
        self.handle = ep.ep_layout(self.idx, self.experts, 1, self.counts, self.rank_tokens, self.in_rank, self.offsets,
                                   handle=self.handle)
        ep.ep_dispatch_ex(self.handle, h, self.received, self.T * self.topk, out_dtype=ep.EP_DTYPE_BF16,
                          overlap_layout=True)
        ep.ep_expert_w4(self.received, self.w_up, self.s_up, self.activated, expert_offsets=self.offsets,
                        activation=ep.EP_ACT_SWIGLU)
        ep.ep_expert_w4(self.activated, self.w_down, self.s_down, self.returned, expert_offsets=self.offsets)
        ep.ep_combine(self.handle, self.returned, self.combined, topk_weights=self.weights)
        return x + self.combined

    def step(self, x):
        """The layer's output [T, hidden] for one new token of each sequence."""
        return self.mixture(self.attention(x))


def main() -> None:
    args = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    args.add_argument("--tokens", type=int, default=64)
    args.add_argument("--steps", type=int, default=20)
    a = args.parse_args()
    layer = DecodeLayer(a.tokens, max_len=2 * a.steps + 64)
    x = torch.randn(a.tokens, 2048, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            layer.step(x)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} sequences, {int(layer.seq_lens[0])} tokens each: {start.elapsed_time(end) / a.steps * 1e3:.1f} us a step, "
          f"outputs finite: {bool(out.isfinite().all())}")


if __name__ == "__main__":
    main()
