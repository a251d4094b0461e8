"""Calls with an explicit stream that allocate a workspace or outputs: that
memory must be the stream's own.  Taken from the current stream's pool it could
still be in use by work that waits there, and would be given out there again
while the call runs."""
import numpy as np
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_f32, dev_i32
from tests.serving_ref import verify
from tests.test_gpu_tree_attention import causal, compare, make

pytestmark = pytest.mark.gpu

PAUSE = 100_000_000  # clocks: 50 ms and more


def leave_pending(nbytes):
    """The current stream, after a pause, copies a block of that size that has
    gone back to its pool by then; the copy, which must be all 3."""
    x = torch.full((nbytes,), 3, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(PAUSE)
    return x.clone()


@pytest.mark.parametrize("d", [64, 128])
def test_attention_workspace_belongs_to_the_stream(d):
    T, L = [9, 3], [20011, 5]
    c = make(T, L, 8, 2, d, seed=d, ps=64)
    q, kn, vn, ptr = c["q"].cuda(), c["kn"].cuda(), c["vn"].cuda(), dev_i32(c["indptr"])
    nbytes = B.csgmv_tree_attention_workspace_bytes(c["cache"], 8)
    out, lse = torch.empty_like(q), torch.empty((sum(T), 8), device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = leave_pending(nbytes)
    B.csgmv_tree_attention(q, kn, vn, c["cache"], 0, ptr, out, lse=lse, stream=s)
    # what the current stream allocates next is not the call's workspace
    others = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert (kept == 3).all() and all((o == 255).all() for o in others)
    compare(c, (out, lse), causal(T))
    for _ in range(20):  # both streams at work
        out.fill_(7.0)
        s.wait_stream(torch.cuda.current_stream())
        B.csgmv_tree_attention(q, kn, vn, c["cache"], 0, ptr, out, lse=lse, stream=s)
        others = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    compare(c, (out, lse), causal(T))


def test_verification_outputs_belong_to_the_stream():
    rng = np.random.default_rng(3)
    V, bs, n = 500, 100, 4
    parents = [-1, 0, 0, 1]
    p = rng.random((bs * n, V)).astype(np.float32)
    p /= p.sum(1, keepdims=True)
    tokens = rng.integers(0, V, bs * n)
    au, su = rng.random(bs * n).astype(np.float32), rng.random(bs).astype(np.float32)
    indptr = dev_i32(np.arange(bs + 1) * n)
    tree = B.DraftTree(bs * n, n)
    B.csgmv_build_draft_tree(tree, dev_i32(parents * bs), indptr)
    dp, dt, da, ds = dev_f32(p), dev_i32(tokens), dev_f32(au), dev_f32(su)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = leave_pending(4 * bs * (n + 2))
    index, count, token = B.csgmv_verify_drafts(dp, dt, indptr, tree, da, ds, stream=s)
    torch.cuda.synchronize()
    assert (kept == 3).all() and tree.device_status() == 0
    for b in range(bs):
        path, last = verify(parents, [int(t) for t in tokens[b * n:b * n + n]], p[b * n:b * n + n], None, au[b * n:b * n + n],
                            su[b])
        assert index[b].tolist() == path + [-1] * (n - len(path)) and int(count[b]) == len(path) and int(token[b]) == last
