"""Training steps of a layer with 16-bit experts, every heavy part through the library.

    python examples/train_experts.py [--tokens 4096] [--steps 20]

Forward of a micro-batch of T tokens

  router                        ep_router_topk (logits: a plain matrix product)
  layout, dispatch              ep_layout, ep_dispatch_ex
  experts' gated blocks         ep_expert_ffn (the layout's offsets)
  weighted combine              ep_combine

and backward

  combine                       ep_combine_backward
  experts' gated blocks         ep_expert_ffn_backward (weight gradients in fp32, added up over micro-batches)
  dispatch                      ep_dispatch_backward
  router                        ep_router_topk_backward

Buffers are made once and a micro-batch enqueues work only. main() fits the layer to a fixed random target by plain
gradient steps on fp32 copies of the weights.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_get_dispatch_layout_gb300 as ep  # noqa: E402


class ExpertLayer:
    """Weights, gradients and buffers of one layer for micro-batches of T tokens."""

    def __init__(self, T: int, hidden: int = 2048, inner: int = 1024, experts: int = 32, topk: int = 4, seed: int = 0):
        g = torch.Generator("cuda").manual_seed(seed)
        bf16, f32 = (dict(dtype=d, device="cuda") for d in (torch.bfloat16, torch.float32))
        self.experts = experts

        def weights(*shape):
            return torch.randn(shape, device="cuda", generator=g) / shape[-1] ** 0.5

        # fp32 weights, which the steps change, and the 16-bit ones that the products read
        self.gate, self.w_up, self.w_down = weights(experts, hidden), weights(experts, 2 * inner, hidden), weights(experts, hidden, inner)
        self.up16, self.down16 = self.w_up.bfloat16(), self.w_down.bfloat16()
        self.grad_gate, self.grad_up, self.grad_down = (torch.zeros_like(w) for w in (self.gate, self.w_up, self.w_down))

        rows = T * topk
        self.logits, self.grad_logits = (torch.empty(T, experts, **f32) for _ in range(2))
        self.idx = torch.empty(T, topk, dtype=torch.int64, device="cuda")
        self.weights, self.grad_weights = (torch.empty(T, topk, **f32) for _ in range(2))
        self.offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
        self.counts = torch.empty(experts, dtype=torch.int32, device="cuda")
        self.ranks = torch.empty(1, dtype=torch.int32, device="cuda")
        self.in_rank = torch.empty(T, 1, dtype=torch.uint8, device="cuda")
        self.handle = None
        self.received, self.returned, self.grad_rows = (torch.empty(rows, hidden, **bf16) for _ in range(3))
        self.gate_up, self.grad_gate_up = (torch.empty(rows, 2 * inner, **bf16) for _ in range(2))
        self.act = torch.empty(rows, inner, **bf16)
        self.out, self.grad_x = (torch.empty(T, hidden, **bf16) for _ in range(2))

    def forward(self, x):
        """x [T, hidden] bf16; the result is the layer's own buffer."""
        self.x = x
        torch.mm(x.float(), self.gate.t(), out=self.logits)
        ep.ep_router_topk(self.logits, self.idx, self.weights, renormalize=True)
        self.handle = ep.ep_layout(self.idx, self.experts, 1, self.counts, self.ranks, self.in_rank, self.offsets, handle=self.handle)
        ep.ep_dispatch_ex(self.handle, x, self.received, len(self.received), out_dtype=ep.EP_DTYPE_BF16)
        ep.ep_expert_ffn(self.received, self.up16, self.down16, self.act, self.returned, gate_up=self.gate_up, expert_offsets=self.offsets)
        ep.ep_combine(self.handle, self.returned, self.out, topk_weights=self.weights)
        return self.out

    def backward(self, grad_out, add: bool = False):
        """Gradients from grad_out [T, hidden] bf16 of the last forward; returns that of x. With `add` the weights' are
        added to those of the micro-batches before."""
        ep.ep_combine_backward(self.handle, grad_out, self.returned, grad_y=self.grad_rows, topk_weights=self.weights,
                               grad_topk_weights=self.grad_weights)
        # the received rows' gradient may take the place of the experts' outputs, which nothing reads any more
        ep.ep_expert_ffn_backward(self.grad_rows, self.received, self.gate_up, self.act, self.up16, self.down16, self.grad_gate_up,
                                  grad_x=self.returned, grad_w_gate_up=self.grad_up, grad_w_down=self.grad_down,
                                  expert_offsets=self.offsets, accumulate=add)
        ep.ep_dispatch_backward(self.handle, self.returned, self.grad_x)
        ep.ep_router_topk_backward(self.logits, self.idx, self.grad_weights, self.grad_logits, renormalize=True)
        self.grad_gate.addmm_(self.grad_logits.t(), self.x.float(), beta=float(add))   # (with 0 what was there does not count, NaN either)
        self.grad_x += (self.grad_logits @ self.gate).bfloat16()
        return self.grad_x

    def step(self, rate: float):
        for w, grad in ((self.gate, self.grad_gate), (self.w_up, self.grad_up), (self.w_down, self.grad_down)):
            w.sub_(grad, alpha=rate)
        self.up16.copy_(self.w_up)
        self.down16.copy_(self.w_down)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inner", type=int, default=1024)
    a = p.parse_args()
    layer = ExpertLayer(a.tokens, a.hidden, a.inner)
    g = torch.Generator("cuda").manual_seed(1)
    batches = [torch.randn(a.tokens, a.hidden, device="cuda", generator=g).bfloat16() for _ in range(2)]
    targets = [torch.tanh(x.flip(1).float()) * 0.3 for x in batches]
    losses = []
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        loss = 0.0
        for k, (x, target) in enumerate(zip(batches, targets)):
            off = layer.forward(x).float() - target
            layer.backward(off.bfloat16(), add=k > 0)
            loss = loss + off.square().mean()
        layer.step(0.3 / a.tokens)
        losses.append(loss)
    torch.cuda.synchronize()
    took = (time.perf_counter() - start) / a.steps
    print(f"{len(batches)} micro-batches of {a.tokens} tokens, {layer.experts} experts: {took * 1e3:.2f} ms a step")
    print("losses", " ".join(f"{v.item():.4f}" for v in losses))
    print("gradients finite:", all(bool(t.isfinite().all()) for t in (layer.grad_gate, layer.grad_up, layer.grad_down, layer.grad_x)))
    layer.handle.destroy()


if __name__ == "__main__":
    main()
