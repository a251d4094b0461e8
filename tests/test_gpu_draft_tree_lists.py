"""Child lists that no tree has: a node under two parents.  Which of them it is
taken for would differ from one CTA of the request's cluster to the next, so the
request is left out; lists that merely end early are walked as far as they go."""
import numpy as np
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_f32, dev_i32
from tests.serving_ref import verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("V", [64, 20000])  # one CTA a request; eight
@pytest.mark.parametrize("n,changes", [
    (4, dict(first_child={1: 2})),  # 2 follows 1 under the root and is 1's child too
    (4, dict(next_sibling={1: 3, 2: 3})),  # two lists run into one
    (200, dict(first_child={150: 199})),  # parents in different warps
])
def test_a_node_under_two_parents_is_left_out(n, changes, V, sampled):
    rng = np.random.default_rng(V + n)
    parents = {4: [-1, 0, 0, 1], 200: list(range(-1, 199))}[n]
    trees = [[-1, 0, 0, 1], parents, [-1, 0, 1]]
    if n == 4 and "next_sibling" in changes:
        trees[1] = [-1, 0, 0, 0]
        changes = dict(next_sibling={1: 2, 2: 3}, first_child={1: 3})
    sizes = [len(t) for t in trees]
    N = sum(sizes)
    indptr = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    tree = B.DraftTree(N, max(sizes))
    B.csgmv_build_draft_tree(tree, dev_i32(sum(trees, [])), dev_i32(indptr))
    for name, put in changes.items():
        for node, to in put.items():
            getattr(tree, name)[4 + node] = to
    p = rng.random((N, V)).astype(np.float32)
    p /= p.sum(1, keepdims=True)
    q = rng.random((N, V)).astype(np.float32)
    q /= q.sum(1, keepdims=True)
    tokens = rng.integers(0, V, N)
    au, su = rng.random(N).astype(np.float32), rng.random(3).astype(np.float32)
    for _ in range(5):
        out = B.csgmv_verify_drafts(dev_f32(p), dev_i32(tokens), dev_i32(indptr), tree, dev_f32(au), dev_f32(su),
                                    draft_probs=dev_f32(q) if sampled else None)
        index, count, token = (t.cpu().numpy() for t in out)
        assert tree.device_status() == 16
        assert count[1] == 0 and token[1] == -1 and (index[1] == -1).all()
        for b in (0, 2):
            a, z = indptr[b], indptr[b + 1]
            path, last = verify(trees[b], [int(t) for t in tokens[a:z]], p[a:z], q[a:z] if sampled else None, au[a:z], su[b])
            assert index[b, :count[b]].tolist() == path and token[b] == last


def test_lists_that_end_early():
    tree = B.DraftTree(4, 4)
    ptr = dev_i32([0, 4])
    B.csgmv_build_draft_tree(tree, dev_i32([-1, 0, 0, 1]), ptr)
    tree.next_sibling[1] = 1  # not above its own number
    tree.first_child[1] = 9  # past the request
    p = torch.zeros((4, 8), device="cuda")
    p[:, 3] = 1.0
    u = torch.zeros(4, device="cuda")
    index, count, token = B.csgmv_verify_drafts(p, dev_i32([0, 3, 3, 3]), ptr, tree, u, u[:1])
    assert tree.device_status() == 0 and index[0].tolist() == [0, 1, -1, -1] and int(count[0]) == 2 and int(token[0]) == 3
