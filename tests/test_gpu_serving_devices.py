"""Serving calls whose operands, stream and current device are not one GPU are
refused before anything is launched.  (With one GPU: the cache and the tree are
made to say that they are on another.)"""
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_i32

pytestmark = pytest.mark.gpu


def calls(cache, tree, stream=None):
    """Every serving call, on operands that are right."""
    q = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    ptr, one, two = dev_i32([0, 2]), dev_i32([0]), dev_i32([1])
    probs, u = torch.full((2, 8), 0.125, device="cuda"), torch.full((2,), 0.5, device="cuda")
    ws = torch.empty(B.csgmv_tree_attention_workspace_bytes(cache, 2), dtype=torch.uint8, device="cuda")
    return [
        lambda: B.csgmv_tree_attention(q, kv[0], kv[0], cache, 0, ptr, torch.empty_like(q), workspace=ws, stream=stream),
        lambda: B.csgmv_kv_commit(cache, kv, kv, None, dev_i32([2]), ptr, stream=stream),
        lambda: B.csgmv_kv_fork(cache, one, two, stream=stream),
        lambda: B.csgmv_kv_copy_pages(cache, one, two, stream=stream),
        lambda: B.csgmv_kv_free(cache, two, stream=stream),
        lambda: B.csgmv_kv_compact(cache, stream=stream),
        lambda: B.csgmv_build_draft_tree(tree, dev_i32([-1, 0]), ptr, stream=stream),
        lambda: B.csgmv_verify_drafts(probs, dev_i32([0, 1]), ptr, tree, u, u[:1], stream=stream),
    ]


def make():
    return B.KvCache.allocate(1, 4, 16, 1, 64, 2, 2), B.DraftTree(2, 2)


def state(cache):
    return [t.clone() for t in (cache.page_table, cache.seq_lens, cache.page_refs)]


def test_operands_of_another_device(monkeypatch):
    cache, tree = make()
    before = state(cache)
    cache.device = tree.device = 1
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in calls(cache, tree)[:5] + calls(cache, tree)[6:]:  # (compaction has no operands but the cache)
        with pytest.raises(B.CsgmvError, match="device|cuda:1"):
            call()
    assert all(torch.equal(a, b) for a, b in zip(before, state(cache)))


def test_another_current_device(monkeypatch):
    cache, tree = make()
    before = state(cache)
    todo = calls(cache, tree)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in todo:
        with pytest.raises(B.CsgmvError, match="current device is cuda:1"):
            call()
    assert all(torch.equal(a, b) for a, b in zip(before, state(cache)))


def test_a_stream_of_another_device():
    class Other:
        device_index, cuda_stream = 1, 0

    cache, tree = make()
    todo = calls(cache, tree, Other())
    todo[-1] = lambda: B._raw_stream(Other(), tree.device)  # (its outputs are allocated on the stream before)
    for call in todo:
        with pytest.raises(B.CsgmvError, match="the stream is on cuda:1"):
            call()


def test_host_tensors_and_workspaces_that_are_not_memory():
    cache, tree = make()
    q = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    ptr = dev_i32([0, 2])
    n = B.csgmv_tree_attention_workspace_bytes(cache, 2)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)):
        with pytest.raises(B.CsgmvError, match="workspace"):
            B.csgmv_tree_attention(q, kv, kv, cache, 0, ptr, torch.empty_like(q), workspace=ws)
    with pytest.raises(B.CsgmvError, match="tree_indptr"):
        B.csgmv_tree_attention(q, kv, kv, cache, 0, ptr.cpu(), torch.empty_like(q))
    for call in calls(cache, tree):  # and what is right runs
        call()
    torch.cuda.synchronize()
    assert cache.device_status() == 0 and tree.device_status() == 0


def test_a_stream_that_is_only_a_handle():
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    cache, tree = make()
    s = torch.cuda.Stream()
    todo = calls(cache, tree, Handle(s))[:7]  # (what allocates outputs needs torch's own)
    s.wait_stream(torch.cuda.current_stream())
    for call in todo:
        call()
    torch.cuda.synchronize()
    assert cache.device_status() == 0 and tree.device_status() == 0
