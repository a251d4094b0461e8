"""Draft trees and their verification against plain references: whole numbers,
so every output is equal."""
import numpy as np
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_f32, dev_i32
from tests.serving_ref import pack_bits, tree_bits, verify

pytestmark = pytest.mark.gpu


def random_tree(rng, n, fan):
    par = [-1]
    for i in range(1, n):
        par.append(int(rng.integers(max(0, i - fan), i)))
    return par[:n]


def build(trees, max_draft, bad=False):
    parents = [p for t in trees for p in t]
    indptr = np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int32)
    tree = B.DraftTree(max(1, len(parents)), max_draft)
    B.csgmv_build_draft_tree(tree, dev_i32(parents), dev_i32(indptr))
    torch.cuda.synchronize()
    return tree, indptr


@pytest.mark.parametrize("sizes,max_draft", [([1], 1), ([5, 0, 1, 32], 32), ([33, 64, 2], 64), ([256, 200, 7], 256)])
def test_derived_fields(sizes, max_draft):
    rng = np.random.default_rng(max_draft)
    trees = [random_tree(rng, n, 6) for n in sizes]
    trees[0] = list(range(-1, sizes[0] - 1))  # a chain
    tree, indptr = build(trees, max_draft)
    assert tree.device_status() == 0
    for b, t in enumerate(trees):
        a, z = indptr[b], indptr[b + 1]
        if a == z:
            continue
        see = tree_bits(t)
        assert np.array_equal(tree.mask[a:z].cpu().numpy(), pack_bits(see, tree.words))
        assert tree.depth[a:z].tolist() == (see.sum(1) - 1).tolist()
        assert tree.first_child[a:z].tolist() == [next((j for j in range(len(t)) if t[j] == i), -1) for i in range(len(t))]
        assert tree.next_sibling[a:z].tolist() == [
            next((j for j in range(i + 1, len(t)) if i > 0 and t[j] == t[i]), -1) for i in range(len(t))]


@pytest.mark.parametrize("bad", [[-1, 0, 3, 1], [0, 0], [-1, -1], [-1, 1], [-1] + [0] * 32])
def test_bad_trees_are_left_out(bad):
    tree, indptr = build([[-1, 0, 0], bad, [-1, 0]], 32)
    assert tree.device_status() == 16
    a, z = indptr[1], indptr[2]
    assert (tree.mask[a:z] == 0).all() and (tree.first_child[a:z] == -1).all() and (tree.next_sibling[a:z] == -1).all()
    assert tree.first_child[:3].tolist() == [1, -1, -1] and tree.first_child[z:z + 2].tolist() == [1, -1]


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def run(trees, tokens, target, draft, au, su, max_draft=None, width=None):
    max_draft = max_draft or max(len(t) for t in trees)
    tree, indptr = build(trees, max_draft)
    idx = None if width is None else torch.full((len(trees), width), 77, dtype=torch.int32, device="cuda")
    out = B.csgmv_verify_drafts(target, dev_i32(tokens), dev_i32(indptr), tree, dev_f32(au), dev_f32(su),
                                draft_probs=draft, accept_index=idx)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out], tree, indptr


def check(trees, tokens, target, draft, au, su):
    (index, count, token), tree, indptr = run(trees, tokens, dev_f32(target), None if draft is None else dev_f32(draft), au, su)
    assert tree.device_status() == 0
    for b, t in enumerate(trees):
        a, z = indptr[b], indptr[b + 1]
        if a == z:
            assert count[b] == 0 and token[b] == -1 and (index[b] == -1).all()
            continue
        path, last = verify(t, [int(x) for x in tokens[a:z]], target[a:z], None if draft is None else draft[a:z], au[a:z],
                            su[b])
        assert index[b].tolist() == path + [-1] * (index.shape[1] - len(path)), b
        assert count[b] == len(path) and token[b] == last, b


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("V,sizes,fan,peak", [
    (1, [2, 1], 1, 1.0), (7, [6, 0, 3, 9], 3, 1.0), (130, [12] * 9, 4, 2.0), (1023, [5, 16, 1, 8] * 3, 3, 4.0),
    (4100, [7] * 5, 2, 5.0), (32001, [6, 9], 3, 5.0)])
def test_walks(V, sizes, fan, peak, sampled):
    rng = np.random.default_rng(V + sampled)
    trees = [random_tree(rng, n, fan) for n in sizes]
    N = sum(sizes)
    logits = rng.normal(size=(N, V)) * peak
    target, draft = softmax(logits), softmax(logits + rng.normal(size=(N, V)) * 0.7)
    base = np.concatenate([[a] * n for a, n in zip(np.cumsum([0] + sizes), sizes) if n]).astype(int)
    par = np.array([max(p, 0) for t in trees for p in t])
    if sampled:
        tokens = np.array([rng.choice(V, p=draft[r].astype(np.float64) / draft[r].sum(dtype=np.float64)) for r in base + par])
    else:  # likely tokens, some of them twice among siblings
        order = np.argsort(-draft, 1)[:, :max(1, min(V, 3))]
        tokens = np.array([order[r, int(rng.integers(0, order.shape[1]))] for r in base + par])
    for trial in range(3):
        au, su = rng.random(N).astype(np.float32), rng.random(len(sizes)).astype(np.float32)
        if trial == 2:  # the ends of the range
            au[:] = 0.0 if V % 2 else np.float32(1) - np.float32(2.0 ** -24)
            su[:] = np.float32(1) - np.float32(2.0 ** -24)
        check(trees, tokens, target, draft if sampled else None, au, su)


def test_equal_distributions_accept_and_unequal_leave_the_rest():
    V = 300
    p = softmax(np.random.default_rng(0).normal(size=(2, V)))
    au, su = np.array([0.5, 0.999], np.float32), np.array([0.3], np.float32)
    (index, count, _), _, _ = run([[-1, 0]], [0, 5], dev_f32(p), dev_f32(p), au, su)
    assert count[0] == 2 and index[0].tolist() == [0, 1]
    # no overlap: the draft is refused and the rest is the target itself
    t, d = np.zeros((2, V), np.float32), np.zeros((2, V), np.float32)
    t[:, 7], t[:, 299], d[:, 3] = 0.25, 0.75, 1.0
    check([[-1, 0]], [0, 3], t, d, au, su)
    # the target is inside the draft's one token: nothing left, so the target itself
    t[:], d[:] = 0.0, 0.0
    t[:, 9], d[:, 9] = 1.0, 1.0
    check([[-1, 0]], [0, 8], t, d, au, su)


def test_rows_with_strides_and_empty_distribution():
    V = 130
    p = softmax(np.random.default_rng(1).normal(size=(6, V)) * 2)
    wide = torch.zeros((6, V + 7), dtype=torch.float32, device="cuda")
    wide[:, :V] = dev_f32(p)
    trees, tok = [[-1, 0, 1], [-1, 0, 0]], [0, 4, 9, 0, 4, 9]
    au, su = np.full(6, 0.4, np.float32), np.array([0.9, 0.1], np.float32)
    (i1, c1, t1), _, _ = run(trees, tok, wide[:, :V], None, au, su)
    (i2, c2, t2), _, _ = run(trees, tok, dev_f32(p), None, au, su)
    assert np.array_equal(i1, i2) and np.array_equal(c1, c2) and np.array_equal(t1, t2)
    wide[3, :V] = 0
    wide[3, 5] = float("nan")  # not a probability: no mass
    (_, c3, t3), tree, _ = run(trees, tok, wide[:, :V], None, au, su)
    assert tree.device_status() == 32 and t3[1] == -1 and c3[1] == 1 and t3[0] == t1[0]


def test_bad_tokens_and_narrow_outputs():
    V = 64
    p = np.full((4, V), 1.0 / V, np.float32)
    au, su = np.zeros(4, np.float32), np.array([0.0], np.float32)
    (index, count, token), tree, _ = run([[-1, 0, 1, 2]], [0, 1, V, 2], dev_f32(p), dev_f32(p), au, su)
    assert tree.device_status() == 32 and count[0] == 2 and index[0].tolist() == [0, 1, -1, -1]
    (index, count, token), tree, _ = run([[-1, 0, 1, 2]], [0, 1, 3, 2], dev_f32(p), dev_f32(p), au, su, width=3)
    assert tree.device_status() == 4 and count[0] == 0 and token[0] == -1 and (index == -1).all()


def test_full_vocabulary_twice_the_same():
    """A serving batch at 128256 tokens: two runs give the same, and the
    sampled tokens have mass in the target."""
    rng = np.random.default_rng(3)
    V, sizes = 128256, [9] * 12
    trees = [random_tree(rng, n, 3) for n in sizes]
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    logits = torch.randn((108, V), generator=g, device="cuda") * 5
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits + torch.randn((108, V), generator=g, device="cuda"), -1)
    tok = rng.integers(0, V, 108)
    au, su = rng.random(108).astype(np.float32), rng.random(12).astype(np.float32)
    a, tree, _ = run(trees, tok, target, draft, au, su)
    b, _, _ = run(trees, tok, target, draft, au, su)
    assert tree.device_status() == 0
    for x, y in zip(a, b):
        assert np.array_equal(x, y)
    for i in range(12):
        path, last = a[0][i][:a[1][i]], a[2][i]
        assert float(target[9 * i + int(path[-1]), int(last)]) > 0


def test_refusals():
    p = torch.full((2, 8), 0.125, device="cuda")
    tree = B.DraftTree(2, 2)
    two, ptr, u, s = dev_i32([0, 1]), dev_i32([0, 2]), dev_f32([0.5, 0.5]), dev_f32([0.5])
    B.csgmv_build_draft_tree(tree, dev_i32([-1, 0]), ptr)
    with pytest.raises(B.CsgmvError, match="target_probs"):
        B.csgmv_verify_drafts(p.half(), two, ptr, tree, u, s)
    with pytest.raises(B.CsgmvError, match="draft_probs"):
        B.csgmv_verify_drafts(p, two, ptr, tree, u, s, draft_probs=p[:, :7])
    with pytest.raises(B.CsgmvError, match="stride"):
        B.csgmv_verify_drafts(p[0].expand(2, 8), two, ptr, tree, u, s)
    with pytest.raises(B.CsgmvError, match="nodes exceed"):
        B.csgmv_build_draft_tree(B.DraftTree(1, 2), dev_i32([-1, 0]), ptr)
    with pytest.raises(B.CsgmvError, match="mask_words"):
        B.csgmv_build_draft_tree(B.DraftTree(2, 300), dev_i32([-1, 0]), ptr)
    assert tree.device_status() == 0
