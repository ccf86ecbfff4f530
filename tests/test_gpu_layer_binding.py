"""The layer operators' binding on a GPU: tensors that are not where a call
expects them, against the same call on ordinary ones."""
import pytest
import torch

from test_gpu_layer import attention_inputs, check_experts, ep, experts_inputs  # noqa: F401  (ep: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3, 24])
def test_experts_take_their_rows_from_pinned_memory(ep, rows):
    """The workspace that the call allocates is the GPU's, wherever x lies."""
    x, w, s, z, off = experts_inputs(rows, [rows - 1, 1], 256, 64, 64, torch.bfloat16, True)
    want = check_experts(ep, x, w, s, z, off, 64)
    pinned = x.cpu().pin_memory()
    y = torch.empty_like(want)
    ep.ep_expert_w4(pinned, w, s, y, expert_offsets=off, zeros=z)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_a_block_table_shared_by_expansion_is_refused(ep):
    q, kc, vc, table, lens = attention_inputs(3, [40, 40], 4, 2, 64, 16, torch.bfloat16)
    work = torch.empty(max(1, ep.ep_paged_attention_workspace(q, kc, table)), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        ep.ep_paged_attention(q, kc, vc, table[:1].expand(2, -1), lens, torch.empty_like(q), work)


def test_tensors_on_another_gpu_than_the_current_one_are_refused(ep, monkeypatch):
    from torch._subclasses import fake_tensor

    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda *a: None)   # (the GPU need not exist)
    with fake_tensor.FakeTensorMode():   # tensors that say where they are and have no memory
        logits, idx = torch.empty(4, 8, device="cuda:1"), torch.empty(4, 2, dtype=torch.int64, device="cuda:1")
        w = torch.empty(4, 2, device="cuda:1")
    with pytest.raises(ValueError, match="current device is cuda:0"):
        ep.ep_router_topk(logits, idx, w)
