"""The paged cache's calls against a host model of the cache: every bit of the
pools and of the bookkeeping."""
import numpy as np
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_i32
from tests.serving_ref import Pool

pytestmark = pytest.mark.gpu


def bits_to_dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(dtype)


def upload(m: Pool, layout="HND", dtype=torch.bfloat16):
    """The model's cache on the device."""
    k, v = (bits_to_dev(x if layout == "NHD" else x.transpose(0, 1, 3, 2, 4), dtype) for x in (m.k, m.v))
    return B.KvCache(k, v, dev_i32(m.table), dev_i32(m.lens), dev_i32(m.refs), layout=layout)


def check(c: B.KvCache, m: Pool, status=0, untouched_free=True):
    torch.cuda.synchronize()
    assert c.device_status() == status
    for t, want, what in ((c.seq_lens, m.lens, "seq_lens"), (c.page_refs, m.refs, "page_refs"),
                          (c.page_table, m.table, "page_table")):
        assert np.array_equal(t.cpu().numpy(), want), what
    for t, want, what in ((c.k_pages, m.k, "k"), (c.v_pages, m.v, "v")):
        got = t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
        got = got if c.layout == "NHD" else got.transpose(0, 1, 3, 2, 4)
        assert np.array_equal(got, want), what


def new_rows(m, n, seed):
    L, _, _, H, D = m.k.shape
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 1 << 16, size=(L, n, H, D)).astype(np.uint16) for _ in range(2))


def commit(c, m, lens, count, index=None, slots=None, seed=1, ok=True):
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = new_rows(m, int(indptr[-1]), seed)
    B.csgmv_kv_commit(c, bits_to_dev(k, c.dtype), bits_to_dev(v, c.dtype),
                      None if index is None else dev_i32(index), dev_i32(count), dev_i32(indptr),
                      None if slots is None else dev_i32(slots))
    assert m.commit(k, v, index, count, indptr, slots) == ok


@pytest.mark.parametrize("layout,dtype", [("HND", torch.bfloat16), ("NHD", torch.float16)])
@pytest.mark.parametrize("ps,heads,d,layers", [(8, 1, 8, 1), (16, 3, 64, 2), (64, 2, 128, 3), (16, 8, 128, 1)])
def test_a_life_of_a_cache(layout, dtype, ps, heads, d, layers):
    """Prompts, drafted tokens, forks, cuts with copy on write, ends and
    compaction, one after the other; after each call every bit is compared."""
    m = Pool(layers, 64, ps, heads, d, 12, 8, seed=ps)
    c = upload(m, layout, dtype)
    rng = np.random.default_rng(ps + d)
    lens = [0, 1, ps - 1, ps, ps + 1, 2 * ps, 3 * ps - 1, 5]
    commit(c, m, lens, lens)  # prompts of every length around a page
    check(c, m)
    draft = [6, 1, 9, 3, 12, 2, 7, 4]
    count = [int(rng.integers(0, n + 1)) for n in draft]
    index = np.full((8, 12), -1, np.int32)
    for b, n in enumerate(count):
        index[b, :n] = np.sort(rng.choice(draft[b], n, replace=False))
    commit(c, m, draft, count, index, seed=2)
    check(c, m)
    B.csgmv_kv_fork(c, dev_i32([4, 6, 3]), dev_i32([8, 9, 10]))
    assert m.fork([4, 6, 3], [8, 9, 10])
    check(c, m)
    # cut a fork inside a page it shares, then append to both holders
    keep = [ps // 2, 0, ps // 2 + 1]
    B.csgmv_kv_free(c, dev_i32([8, 1, 9]), dev_i32(keep))
    m.free([8, 1, 9], keep)
    check(c, m)
    commit(c, m, [3, 2, 4], [3, 1, 4], slots=[8, 4, 9], seed=3)
    check(c, m)
    B.csgmv_kv_free(c, dev_i32([0, 3, 6]))
    m.free([0, 3, 6])
    check(c, m)
    B.csgmv_kv_compact(c)
    m.compact()
    check(c, m)
    B.csgmv_kv_compact(c)  # nothing left to move
    m.compact()
    check(c, m)


def test_both_holders_of_a_cut_page_append_at_once():
    m = Pool(2, 16, 16, 2, 64, 4, 4)
    c = upload(m)
    commit(c, m, [40], [40])
    B.csgmv_kv_fork(c, dev_i32([0]), dev_i32([1]))
    m.fork([0], [1])
    B.csgmv_kv_free(c, dev_i32([0, 1]), dev_i32([20, 25]))
    m.free([0, 1], [20, 25])
    check(c, m)
    commit(c, m, [5, 30], [5, 30], slots=[1, 0], seed=5)
    check(c, m)
    assert (m.refs[m.table[0, :1]] == 2).all()


@pytest.mark.parametrize("pages,frac", [(1, 1.0), (33, 0.5), (1000, 0.3), (70001, 0.01), (4096, 0.0), (5000, 1.0)])
def test_compaction_of_random_pools(pages, frac):
    """Any pattern of live pages, shared ones among them, odd pool sizes."""
    rng = np.random.default_rng(pages)
    m = Pool(1, pages, 8, 1, 8, 16, max(1, pages // 8))
    live = rng.permutation(pages)[:int(pages * frac)]
    for i, p in enumerate(live):
        s = i % 16
        j = i // 16
        if j >= m.max_pages:
            break
        m.table[s, j] = p
        m.refs[p] = 1
        m.lens[s] = (j + 1) * 8 - (i % 3 if i >= len(live) - 16 else 0)
    if len(live) > 40:  # two more holders of one page
        m.refs[m.table[0, 0]] += 1
        m.table[1, 0], m.refs[m.table[1, 0]] = m.table[0, 0], 0
    c = upload(m)
    B.csgmv_kv_compact(c)
    m.compact()
    check(c, m)
    n = int((m.refs > 0).sum())
    assert (m.refs[:n] > 0).all() and (m.refs[n:] == 0).all()


def test_pages_come_lowest_first_and_run_out_whole():
    """A batch that does not fit leaves everything as it was."""
    m = Pool(1, 6, 16, 1, 64, 4, 6)
    m.refs[[0, 3]] = 1
    c = upload(m)
    commit(c, m, [30, 16], [30, 16])
    check(c, m)
    assert list(m.table[0, :2]) == [1, 2] and m.table[1, 0] == 4
    commit(c, m, [17], [17], slots=[2], ok=False)
    check(c, m, status=4)
    c.status.zero_()
    commit(c, m, [16], [16], slots=[2])
    check(c, m)
    B.csgmv_kv_fork(c, dev_i32([0]), dev_i32([3]))  # 30 tokens: needs a page for its last one
    assert not m.fork([0], [3])
    check(c, m, status=4)


def test_bad_entries_are_left_out():
    m = Pool(1, 32, 16, 1, 64, 6, 2)
    c = upload(m)
    commit(c, m, [20, 5], [20, 5])
    # a slot out of range, a slot twice, a node number out of range, a row of
    # the table too short, a negative count; one sound request between them
    indptr = np.array([0, 4, 8, 12, 16, 36, 40], np.int32)
    k, v = new_rows(m, 40, 9)
    index = np.tile(np.arange(20, dtype=np.int32), (6, 1))
    index[3, 1] = 4
    slots, count = [6, 2, 2, 3, 0, 1], [4, 3, 3, 2, 20, -1]
    B.csgmv_kv_commit(c, bits_to_dev(k, c.dtype), bits_to_dev(v, c.dtype), dev_i32(index), dev_i32(count),
                      dev_i32(indptr), dev_i32(slots))
    m.commit(k, v, index, [0, 3, 0, 0, 0, 0], indptr, [0, 2, 0, 0, 0, 0])
    check(c, m, status=1 | 4 | 8 | 16)
    c.status.zero_()
    # a child in use, a child twice, a child that is a parent, slots out of range
    B.csgmv_kv_fork(c, dev_i32([0, 0, 0, 0, 4, -1]), dev_i32([1, 3, 3, 4, 5, 5]))
    assert m.fork([0], [3])
    check(c, m, status=1)
    c.status.zero_()
    B.csgmv_kv_free(c, dev_i32([9, 1, 0, 0]), dev_i32([0, -2, 16, 7]))
    m.free([0], [7])
    check(c, m, status=1 | 8)


def test_copy_pages_and_another_stream():
    m = Pool(3, 9, 16, 2, 64, 2, 4)
    c = upload(m)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.csgmv_kv_copy_pages(c, dev_i32([0, 4, 9, 2, 7]), dev_i32([8, 1, 3, -1, 7]))
    s.synchronize()
    for pool in (m.k, m.v):
        pool[:, 8], pool[:, 1] = pool[:, 0], pool[:, 4]
    check(c, m, status=2)


def test_strided_pool_and_rows():
    """Pages with room between heads and layers; rows cut from one projection."""
    m = Pool(2, 8, 16, 2, 64, 2, 4)
    big = torch.zeros((2, 9, 3, 16, 72), dtype=torch.bfloat16, device="cuda")
    big2 = torch.zeros_like(big)
    views = [t[:, :8, :2, :, :64] for t in (big, big2)]
    for t, x in zip(views, (m.k, m.v)):
        t.copy_(bits_to_dev(x.transpose(0, 1, 3, 2, 4), torch.bfloat16))
    c = B.KvCache(*views, dev_i32(m.table), dev_i32(m.lens), dev_i32(m.refs))
    rows = torch.randn((2, 20, 6, 64), device="cuda").bfloat16()
    k, v = rows[:, :, 1:3], rows[:, :, 4:6]
    B.csgmv_kv_commit(c, k, v, None, dev_i32([9, 11]), dev_i32([0, 9, 20]))
    kb, vb = (t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16) for t in (k, v))
    m.commit(kb, vb, None, [9, 11], [0, 9, 20])
    check(c, m)
    assert int(big[:, 8].abs().sum()) == 0 and int(big[:, :, 2].abs().sum()) == 0


def test_pool_beyond_32_bit_offsets():
    """Pages whose element offsets pass 2^31."""
    pages = (1 << 31) // (16 * 8 * 128) + 64
    c = B.KvCache.allocate(1, pages, 16, 8, 128, 2, 8)
    c.page_refs[:pages - 4] = 1
    rows = torch.randn((1, 40, 8, 128), device="cuda").bfloat16()
    B.csgmv_kv_commit(c, rows, rows, None, dev_i32([40]), dev_i32([0, 40]))
    B.csgmv_kv_fork(c, dev_i32([0]), dev_i32([1]))
    torch.cuda.synchronize()
    assert c.device_status() == 0
    assert c.page_table[0, :3].tolist() == [pages - 4, pages - 3, pages - 2]
    assert c.page_table[1, :3].tolist() == [pages - 4, pages - 3, pages - 1]
    for s in (0, 1):
        got = c.k_pages[0, c.page_table[s, :3].long()].transpose(1, 2).reshape(48, 8, 128)[:40]
        assert torch.equal(got, rows[0])


def test_refusals():
    c = B.KvCache.allocate(1, 4, 16, 1, 64, 2, 2)
    rows = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    one, ptr = dev_i32([1]), dev_i32([0, 4])
    with pytest.raises(B.CsgmvError, match="type"):
        B.csgmv_kv_commit(c, rows.half(), rows.half(), None, one, ptr)
    with pytest.raises(B.CsgmvError, match="layers"):
        B.csgmv_kv_commit(c, rows.repeat(2, 1, 1, 1), rows.repeat(2, 1, 1, 1), None, one, ptr)
    with pytest.raises(B.CsgmvError, match="accept_len"):
        B.csgmv_kv_commit(c, rows, rows, None, one.long(), ptr)
    with pytest.raises(B.CsgmvError, match="max_seqs"):
        B.csgmv_kv_free(c, dev_i32([0, 1, 0]))
    with pytest.raises(B.CsgmvError, match="page_size"):
        B.csgmv_kv_compact(B.KvCache.allocate(1, 4, 12, 1, 64, 2, 2))
    with pytest.raises(B.CsgmvError, match="layout"):
        B.KvCache.allocate(1, 4, 16, 1, 64, 2, 2, layout="DHN")
    assert c.device_status() == 0
