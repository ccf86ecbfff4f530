"""CPU-only checks of the layer operators' binding: what it refuses before the
library is called. No tensor here has an address that a kernel could use."""
import pytest
import torch


@pytest.fixture(scope="module")
def ep():
    from combine_get_dispatch_layout_gb300.build import build
    import combine_get_dispatch_layout_gb300 as ep

    build()
    ep.lib()
    return ep


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype)


def attend(ep, **kw):
    cache = empty(0, 8, 1, 0)
    a = dict(q=empty(2, 1, 0), k_cache=cache, v_cache=cache, block_table=empty(2, 0, dtype=torch.int32),
             seq_lens=empty(0, dtype=torch.int32), out=empty(2, 1, 0), workspace=empty(0, dtype=torch.uint8), stream=0)
    ep.ep_paged_attention(**{**a, **kw})


@pytest.mark.parametrize("table", [torch.zeros(1, 3, dtype=torch.int32).expand(2, 3),
                                   torch.zeros(8, dtype=torch.int32).as_strided((2, 3), (2, 1))])
def test_rows_of_a_block_table_that_overlap_are_refused(ep, table):
    """One table for all sequences, by expand(), has rows no distance apart: the kernel would read past it."""
    with pytest.raises(ValueError, match="overlap"):
        attend(ep, block_table=table)


def test_other_rows_that_overlap_are_refused(ep):
    idx, w = empty(2, 1, dtype=torch.int64), empty(2, 1, dtype=torch.float32)
    with pytest.raises(ValueError, match="overlap"):
        ep.ep_router_topk(empty(1, 8).expand(2, 8), idx, w, stream=0)


def test_a_workspace_of_the_host_is_refused(ep):
    """Kernels that run after the call write it, and address it by tensor maps."""
    with pytest.raises(ValueError, match="workspace"):
        ep.ep_expert_w4(empty(0, 128), empty(0, 8, 64, dtype=torch.uint8), empty(0, 1, 8), empty(0, 8),
                        workspace=empty(0, dtype=torch.uint8), stream=0)


def test_tensors_on_two_gpus_are_refused(ep, monkeypatch):
    from torch._subclasses import fake_tensor

    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda *a: None)   # (the GPUs need not exist)
    with fake_tensor.FakeTensorMode():   # tensors that say where they are and have no memory
        logits = torch.empty(4, 8, device="cuda:1")
        idx, w = torch.empty(4, 2, dtype=torch.int64, device="cuda:0"), torch.empty(4, 2, device="cuda:0")
    with pytest.raises(ValueError, match="cuda:1 and on cuda:0"):
        ep.ep_router_topk(logits, idx, w, stream=0)


def test_an_option_without_a_truth_value_is_refused_before_the_call(ep):
    logits, idx, w = empty(0, 8), empty(0, 2, dtype=torch.int64), empty(0, 2, dtype=torch.float32)
    ep.ep_router_topk(logits, idx, w, stream=0)
    for call in (lambda o: ep.ep_router_topk(logits, idx, w, renormalize=o, stream=0),
                 lambda o: ep.ep_router_topk_backward(logits, idx, w, logits, renormalize=o, stream=0)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call(torch.tensor([1, 1]))
