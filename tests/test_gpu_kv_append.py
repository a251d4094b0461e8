"""csgmv_kv_extend and csgmv_kv_append: slots and bookkeeping against lists of
pages, contents against float64, and both against csgmv_kv_commit.  What is not
appended stays as it is."""
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.step_ref import Cache, close, rotary

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
BAD_SEQ, BAD_PAGE, CAPACITY, BAD_LENS = 1, 2, 4, 8


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def make(lens, ps=16, layers=2, heads=2, d=64, dtype=BF, layout="HND", spare=12, width=None, seed=0, share=()):
    """A cache whose sequences hold `lens` tokens on scattered pages of random
    values; share: (sequence, its copy by a fork)."""
    g = torch.Generator().manual_seed(seed)
    width = width or max(-(-n // ps) for n in lens) + 8
    pages = sum(-(-n // ps) for n in lens) + spare
    c = B.KvCache.allocate(layers, pages, ps, heads, d, len(lens), width, dtype=dtype, layout=layout)
    order = torch.randperm(pages, generator=g).tolist()
    refs = [0] * pages
    for s, n in enumerate(lens):
        for i in range(-(-n // ps)):
            c.page_table[s, i] = order.pop()
            refs[int(c.page_table[s, i])] = 1
    for a, b in share:  # b holds a's pages too
        c.page_table[b] = c.page_table[a]
        for i in range(-(-lens[a] // ps)):
            refs[int(c.page_table[a, i])] += 1
    c.page_refs.copy_(ints(refs))
    c.seq_lens.copy_(ints([lens[dict((b, a) for a, b in share).get(s, s)] for s in range(len(lens))]))
    for pool in (c.k_pages, c.v_pages):
        pool.copy_(torch.randn(pool.shape, generator=g))
    return c, g


def rows(pool, layout):
    """(layers, pages * page_size, heads, d)"""
    t = pool if layout == "NHD" else pool.transpose(2, 3)
    return t.flatten(1, 2)


def copy_of(c):
    o = B.KvCache(c.k_pages.clone(), c.v_pages.clone(), c.page_table.clone(), c.seq_lens.clone(), c.page_refs.clone(), layout=c.layout)
    return o


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("ps,d,dtype,rot,interleaved", [(8, 64, BF, 64, False), (16, 128, HF, 128, True), (64, 80, BF, 20, False),
                                                        (128, 8, HF, 4, True), (16, 128, BF, 64, False)])
def test_appended_rows(layout, ps, d, dtype, rot, interleaved):
    lens, add = [0, 1, ps - 1, ps, 3 * ps + 5, 0], [1, ps, 2, 1, 0, 2 * ps + 3]
    c, g = make(lens, ps=ps, d=d, dtype=dtype, layout=layout)
    ref, seqs = Cache(c), [3, 0, 5, 1, 4, 2]
    ptr = [0]
    for s in seqs:
        ptr.append(ptr[-1] + add[s])
    n, hq = ptr[-1], 6
    slots, pos = B.csgmv_kv_extend(c, ints(ptr), n, seq_slots=ints(seqs))
    want, at = [], []
    for s in seqs:
        at += range(ref.lens[s], ref.lens[s] + add[s])
        got, copies = ref.extend(s, add[s])
        want += got
        assert not copies
    assert slots.tolist() == want and pos.tolist() == at and c.device_status() == 0
    assert (c.page_table.tolist(), c.seq_lens.tolist(), c.page_refs.tolist()) == (ref.table, ref.lens, ref.refs)
    rope = B.Rope(d, rotary_dim=rot, interleaved=interleaved, scaling=("linear", 2.0))
    for layer in (1, 0):
        qkv = torch.randn((n, (hq + 4) * d), generator=g).to(dtype).cuda()
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([hq * d, 2 * d, 2 * d], 1))
        kp, vp = rows(c.k_pages, layout).clone(), rows(c.v_pages, layout).clone()
        qo, ko = torch.empty((n, hq, d), dtype=dtype, device="cuda"), torch.empty((n, 2, d), dtype=dtype, device="cuda")
        B.csgmv_kv_append(c, layer, k, v, slots, pos, rope=rope, q=q, q_out=qo, k_out=ko if layer else None)
        turned, tol = rotary(k, pos, rope.freq, rot, interleaved)
        close(rows(c.k_pages, layout)[layer, slots], turned, tol)
        assert torch.equal(rows(c.v_pages, layout)[layer, slots], v)
        close(qo, *rotary(q, pos, rope.freq, rot, interleaved))
        if layer:
            assert torch.equal(ko, rows(c.k_pages, layout)[layer, slots])
        kp[layer, slots], vp[layer, slots] = rows(c.k_pages, layout)[layer, slots], v
        assert torch.equal(kp, rows(c.k_pages, layout)) and torch.equal(vp, rows(c.v_pages, layout))


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_the_same_as_a_commit(layout):
    """Without a rope, extend and append leave what a commit of the same rows
    does; shared pages are copied first."""
    lens = [5, 40, 0, 17, 0]
    c, g = make(lens, share=((0, 2), (3, 4)), layout=layout, layers=3)
    other = copy_of(c)
    n, add = 60, [20, 7, 1, 30]
    ptr, seqs = [1, 21, 28, 29, 59], [2, 3, 1, 0]  # rows 0 and 59 are nobody's
    k, v = (torch.randn((3, n, 2, 64), generator=g).to(BF).cuda() for _ in range(2))
    before = torch.empty(5, dtype=torch.int32, device="cuda")
    slots, pos = B.csgmv_kv_extend(c, ints(ptr), n, add_lens=ints(add), seq_slots=ints(seqs), lens_before=before)
    assert before.tolist() == [5, 40, 5, 17, 17]
    assert slots[0] == -1 and slots[59] == -1 and int(pos[0]) == 0
    for layer in range(3):
        B.csgmv_kv_append(c, layer, k[layer], v[layer], slots)
    B.csgmv_kv_commit(other, k, v, None, ints(add), ints(ptr), seq_slots=ints(seqs))
    for a, b in ((c.page_table, other.page_table), (c.seq_lens, other.seq_lens), (c.page_refs, other.page_refs),
                 (c.k_pages, other.k_pages), (c.v_pages, other.v_pages)):
        assert torch.equal(a, b)
    assert c.device_status() == other.device_status() == 0


def test_fewer_tokens_than_rows():
    """add_lens below the rows: the rest of a request's rows have no slot, and
    append leaves their outputs as they are."""
    c, g = make([3, 9])
    slots, pos = B.csgmv_kv_extend(c, ints([0, 4, 10]), 10, add_lens=ints([2, 0]))
    assert (slots >= 0).tolist() == [True, True] + [False] * 8 and pos.tolist() == [3, 4] + [0] * 8
    assert c.seq_lens.tolist() == [5, 9]
    k, q = torch.randn((10, 2, 64), generator=g).to(BF).cuda(), torch.randn((10, 4, 64), generator=g).to(BF).cuda()
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    pools = c.k_pages.clone(), c.v_pages.clone()
    B.csgmv_kv_append(c, 0, k, k, slots, pos, rope=B.Rope(64), q=q, q_out=qo, k_out=ko)
    assert bool((qo[2:] == 7).all()) and bool((ko[2:] == 7).all()) and not bool((qo[:2] == 7).all())
    for pool, was in zip((c.k_pages, c.v_pages), pools):
        new, old = rows(pool, "HND"), rows(was, "HND").clone()
        old[0, slots[:2]] = new[0, slots[:2]]
        assert torch.equal(new, old)


@pytest.mark.parametrize("add,seqs,ptr,status,extended", [
    ([1, 1, 1], [0, 9, 1], [0, 1, 2, 3], BAD_SEQ, [0, 2]), ([1, 1, 1], [0, -1, 1], [0, 1, 2, 3], BAD_SEQ, [0, 2]),
    ([1, 1, 1], [1, 0, 1], [0, 1, 2, 3], BAD_SEQ, [0, 1]), ([1, 2, 1], [0, 1, 2], [0, 1, 2, 3], BAD_LENS, [0, 2]),
    ([1, -1, 1], [0, 1, 2], [0, 1, 2, 3], BAD_LENS, [0, 2]), ([1, 200, 1], [0, 1, 2], [0, 1, 201, 202], CAPACITY, [0, 2]),
    # indptr that is none: nothing
    ([1, 1, 1], [0, 1, 2], [0, 2, 1, 3], BAD_LENS, []), ([1, 1, 1], [0, 1, 2], [-1, 1, 2, 3], BAD_LENS, []),
    ([1, 1, 1], [0, 1, 2], [0, 1, 2, 900], BAD_LENS, [])])
def test_requests_that_are_left_out(add, seqs, ptr, status, extended):
    c, _ = make([5, 20, 0])
    ref, n = Cache(c), 202
    slots, pos = B.csgmv_kv_extend(c, ints(ptr), n, add_lens=ints(add), seq_slots=ints(seqs))
    want, at = [-1] * n, [0] * n
    for b in extended:
        s = seqs[b]
        at[ptr[b]:ptr[b] + add[b]] = range(ref.lens[s], ref.lens[s] + add[b])
        want[ptr[b]:ptr[b] + add[b]] = ref.extend(s, add[b])[0]
    assert c.device_status() & status and slots.tolist() == want and pos.tolist() == at
    assert (c.page_table.tolist(), c.seq_lens.tolist(), c.page_refs.tolist()) == (ref.table, ref.lens, ref.refs)


def test_too_few_pages_extend_nothing():
    c, _ = make([16, 16], spare=3)
    ref = Cache(c)
    before = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    slots, pos = B.csgmv_kv_extend(c, ints([0, 33, 50]), 50, lens_before=before)
    assert c.device_status() == CAPACITY and bool((slots == -1).all()) and not bool(pos.any())
    assert (c.page_table.tolist(), c.seq_lens.tolist(), c.page_refs.tolist()) == (ref.table, ref.lens, ref.refs)
    assert before.tolist() == [16, 16]


def test_a_page_table_with_a_bad_page():
    c, _ = make([5, 20])
    c.page_table[1, 1] = 10 ** 6
    slots, _ = B.csgmv_kv_extend(c, ints([0, 1, 2]), 2)
    assert c.device_status() == BAD_PAGE and slots[1] == -1 and slots[0] >= 0


def test_no_requests():
    c, _ = make([5, 20])
    slots, pos = B.csgmv_kv_extend(c, ints([0]), 3)
    assert slots.tolist() == [-1] * 3 and c.seq_lens.tolist() == [5, 20] and c.device_status() == 0
    before = torch.empty(2, dtype=torch.int32, device="cuda")
    B.csgmv_kv_extend(c, ints([0]), 0, lens_before=before)
    assert before.tolist() == [5, 20]


def test_slots_outside_the_cache_are_left_out():
    c, g = make([5, 20])
    most = c.num_pages * c.page_size
    k = torch.randn((5, 2, 64), generator=g).to(BF).cuda()
    pools = c.k_pages.clone(), c.v_pages.clone()
    B.csgmv_kv_append(c, 1, k, k, ints([-1, -1, -1, -1, -1], torch.int64))
    assert c.device_status() == 0
    B.csgmv_kv_append(c, 1, k, k, ints([most, -2, -1, 2 ** 62, -2 ** 63], torch.int64))
    assert c.device_status() == BAD_PAGE
    assert torch.equal(c.k_pages, pools[0]) and torch.equal(c.v_pages, pools[1])
    B.csgmv_kv_append(c, 1, k, k, ints([-1, most - 1, -1, -1, 0], torch.int64))
    assert torch.equal(rows(c.k_pages, "HND")[1, most - 1], k[1]) and torch.equal(rows(c.v_pages, "HND")[1, 0], k[4])


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_slots_past_32_bits_of_elements(layout):
    """2.2e9 elements a pool: the last slots are where they belong."""
    c = B.KvCache.allocate(1, 34000, 64, 8, 128, 1, 8, layout=layout)
    most, g = c.num_pages * c.page_size, torch.Generator().manual_seed(1)
    k, v = (torch.randn((3, 8, 128), generator=g).to(BF).cuda() for _ in range(2))
    at = [most - 1, most - 64, 5]
    B.csgmv_kv_append(c, 0, k, v, ints(at, torch.int64))
    for i, a in enumerate(at):
        for pool, new in ((c.k_pages, k), (c.v_pages, v)):
            page = pool[0, a // 64]
            assert torch.equal(page[:, a % 64] if layout == "HND" else page[a % 64], new[i])


def test_pages_with_gaps_and_heads_broadcast():
    """Strides of the cache beyond its sizes; one head's values for all heads."""
    wide = torch.full((2, 6, 3, 20, 72), 7.0, dtype=BF, device="cuda"), torch.full((2, 6, 3, 20, 72), 7.0, dtype=BF, device="cuda")
    kp, vp = (w[:, :, :, :16, :64] for w in wide)
    c = B.KvCache(kp, vp, torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                  torch.zeros(6, dtype=torch.int32, device="cuda"))
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn((20, 3, 64), generator=g).to(BF).cuda(), torch.randn((20, 1, 64), generator=g).to(BF).cuda().expand(20, 3, 64)
    slots, pos = B.csgmv_kv_extend(c, ints([0, 17, 20]), 20)
    rope = B.Rope(64, interleaved=True)
    B.csgmv_kv_append(c, 1, k, v, slots, pos, rope=rope)
    close(rows(kp, "HND")[1, slots], *rotary(k, pos, rope.freq, 64, True))
    assert torch.equal(rows(vp, "HND")[1, slots], v)
    for w, p in zip(wide, (kp, vp)):
        p.fill_(7.0)
        assert bool((w == 7.0).all())


def test_keys_turned_in_place():
    """k_out = k: a projection's rows are ready for attention and in the cache."""
    c, g = make([5, 20, 100], d=128, layout="NHD")
    n, rope = 30, B.Rope(128)
    slots, pos = B.csgmv_kv_extend(c, ints([0, 10, 11, 30]), n)
    qkv = torch.randn((n, 8 * 128), generator=g).to(BF).cuda()
    was = qkv.clone()
    q, k, v = (t.unflatten(1, (-1, 128)) for t in qkv.split([512, 256, 256], 1))
    B.csgmv_kv_append(c, 1, k, v, slots, pos, rope=rope, q=q, k_out=k)
    close(q, *rotary(was[:, :512].unflatten(1, (4, 128)), pos, rope.freq, 128, False))
    close(k, *rotary(was[:, 512:768].unflatten(1, (2, 128)), pos, rope.freq, 128, False))
    assert torch.equal(qkv[:, 768:], was[:, 768:])
    assert torch.equal(rows(c.k_pages, "NHD")[1, slots], k) and torch.equal(rows(c.v_pages, "NHD")[1, slots], v)


@pytest.mark.parametrize("rot", [None, 0, 32])
@pytest.mark.parametrize("keys", [False, True])
def test_queries_partly_turned_in_place(rot, keys):
    """What of them is not turned keeps its bits; the keys' is written to the cache."""
    c, g = make([5, 20, 100], d=128, dtype=HF)
    n, rope = 30, None if rot is None else B.Rope(128, rotary_dim=rot)
    turn = rot or 0
    slots, pos = B.csgmv_kv_extend(c, ints([0, 10, 11, 30]), n)
    q, k, v = (torch.randn((n, h, 128), generator=g).to(HF).cuda() for h in (4, 2, 2))
    q.view(torch.int16)[..., turn:] = torch.randint(-2 ** 15, 2 ** 15, (n, 4, 128 - turn), generator=g, dtype=torch.int16).cuda()
    was = q.clone(), k.clone(), v.clone()
    B.csgmv_kv_append(c, 0, k, v, slots, pos, rope=rope, q=q, k_out=k if keys else None)
    for x, y in ((was[0], q), (was[1], rows(c.k_pages, "HND")[0, slots])):
        if turn:
            close(y[..., :turn], *(t[..., :turn] for t in rotary(x.nan_to_num(), pos, rope.freq, turn, False)))
        assert torch.equal(y.view(torch.int16)[..., turn:], x.view(torch.int16)[..., turn:])
    assert torch.equal(k, rows(c.k_pages, "HND")[0, slots] if keys else was[1])
    assert torch.equal(v, was[2]) and torch.equal(rows(c.v_pages, "HND")[0, slots], v)


def test_many_requests_and_empty_ones():
    lens = [i % 37 for i in range(700)]
    c, g = make(lens, ps=8, layers=1, heads=1, d=8, spare=700)
    ref = Cache(c)
    add = [(i * 7) % 5 if i % 3 else 0 for i in range(700)]
    ptr = [0]
    for a in add:
        ptr.append(ptr[-1] + a)
    slots, pos = B.csgmv_kv_extend(c, ints(ptr), ptr[-1] + 4)
    want = [s for b in range(700) for s in ref.extend(b, add[b])[0]]
    assert slots.tolist() == want + [-1] * 4 and c.device_status() == 0
    assert (c.page_table.tolist(), c.page_refs.tolist()) == (ref.table, ref.refs)


def test_a_captured_step_is_replayed():
    """extend and appends in one graph: each replay puts the next token behind."""
    c, g = make([5, 14], layers=2)
    ref, rope, ptr = Cache(c), B.Rope(64), ints([0, 1, 2])
    k, v = (torch.randn((2, 2, 64), generator=g).to(BF).cuda() for _ in range(2))
    slots, pos = torch.empty(2, dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        B.csgmv_kv_extend(c, ptr, 2, slots=slots, positions=pos)
        for layer in range(2):
            B.csgmv_kv_append(c, layer, k, v, slots, pos, rope=rope)
    for _ in range(4):
        k.copy_(torch.randn((2, 2, 64), generator=g))
        graph.replay()
        want = [ref.extend(b, 1)[0][0] for b in range(2)]
        assert slots.tolist() == want
        turned, tol = rotary(k, pos, rope.freq, 64, False)
        for layer in range(2):
            close(rows(c.k_pages, "HND")[layer, slots], turned, tol)
    assert c.seq_lens.tolist() == ref.lens and c.device_status() == 0


def test_the_cache_seen_with_other_lengths():
    c, _ = make([5, 20])
    with pytest.raises(B.CsgmvError):
        c.with_lens(torch.zeros(3, dtype=torch.int32, device="cuda"))
    before = c.seq_lens.clone()
    old = c.with_lens(before)
    B.csgmv_kv_extend(c, ints([0, 2, 4]), 4)
    assert c.seq_lens.tolist() == [7, 22] and old.seq_lens.tolist() == [5, 20] and old.c.seq_lens == before.data_ptr()
    assert old.c.page_table == c.c.page_table and old.c.scratch == c.c.scratch
