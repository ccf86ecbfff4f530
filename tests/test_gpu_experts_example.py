"""The training example's gradients from one step to the next."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def test_a_new_step_forgets_a_micro_batch_of_nan():
    """A step's first micro-batch overwrites the gradients of the step before, whatever they were."""
    import train_experts

    g = torch.Generator().manual_seed(3)
    x, d_out = ((torch.randn(40, 64, generator=g)).bfloat16().cuda() for _ in range(2))
    layer, other = (train_experts.ExpertLayer(40, hidden=64, inner=32, experts=4, topk=2) for _ in range(2))
    layer.forward(x)
    layer.backward(torch.full_like(d_out, math.nan))
    for one in (layer, other):
        one.forward(x)
        one.backward(d_out)
    for a, b in ((layer.grad_gate, other.grad_gate), (layer.grad_up, other.grad_up), (layer.grad_down, other.grad_down)):
        assert torch.equal(a, b) and a.isfinite().all()
    for one in (layer, other):
        one.handle.destroy()
