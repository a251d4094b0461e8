"""Host checks of the serving operators' C calls that keep sizes within what the
kernels' arithmetic holds, and buffers that steer a kernel apart from what it
writes.  CPU only: no kernel runs."""
import ctypes

import pytest

from tests.test_serving_abi import CAPACITY, INVALID, P, UNSUPPORTED, attend, cache, commit, lib  # noqa: F401


def test_rows_of_a_kv_head_fit_30_bits(lib):  # noqa: F811
    most = (1 << 24) - 1
    for n, hq in ((most, 256), (1 << 23, 258 // 2 * 2), (most, 2 * 65)):  # 128, 129 and 65 query heads a kv head
        assert attend(lib, cache(), n=n, hq=hq) == UNSUPPORTED
    assert attend(lib, cache(), n=most, hq=2 * 65) == UNSUPPORTED and b"2^30" in lib.csgmv_last_error()
    # 64 of them fit: refused for the next thing that is wrong
    assert attend(lib, cache(), n=most, hq=2 * 64, q=None) == INVALID and b"NULL" in lib.csgmv_last_error()


@pytest.mark.parametrize("kw,ok", [
    (dict(layer_stride=0), False), (dict(layer_stride=8), False), (dict(layer_stride=2048), False),
    (dict(layer_stride=15 * 2048), False), (dict(layer_stride=16 * 2048), True), (dict(layer_stride=17 * 2048 + 8), True),
    (dict(layer_stride=2048, page_stride=4 * 2048), True),  # layers inside pages
    (dict(layer_stride=2048, page_stride=3 * 2048), False), (dict(layer_stride=2040, page_stride=4 * 2048), False),
    (dict(layer_stride=1024, head_stride=4 * 1024, page_stride=8 * 1024), True),  # inside heads
    (dict(layer_stride=64, token_stride=4 * 64, head_stride=4096, page_stride=8192), True),  # inside tokens
    (dict(layer_stride=0, num_layers=1), True), (dict(layer_stride=8, num_layers=1), True),
    (dict(layer_stride=1 << 62), False),  # past 64 bits
])
def test_layers_of_a_cache_keep_to_themselves(lib, kw, ok):  # noqa: F811
    """Calls copy all layers at once: two layers that share memory would leave
    there whichever comes last."""
    c = cache(**kw)
    # what is right is refused for the next thing: a negative number of requests
    assert commit(lib, c, bs=-1) == INVALID
    assert (b"overlap" in lib.csgmv_last_error()) is not ok


@pytest.mark.parametrize("kw,ok", [
    (dict(), True),
    # written over by one another, or over what the kernels find their way by
    (dict(lse=0x80000000), False), (dict(lse=0x80000000 - 64), False), (dict(lse=0x40000000 + 512), False),
    (dict(lse=P), False), (dict(ws=P - 4096), False), (dict(out=P - 128), False),
    (dict(out=0x50000000 - 64), False), (dict(lse=0x50000000), False), (dict(ws=0x50000000 - 65536), False),
    (dict(lse=0x50000010), True),  # right behind the four slots
    # rows of the output in one another
    (dict(ots=0), False), (dict(ohs=0), False), (dict(ohs=56), False), (dict(ots=504), False), (dict(ots=64, ohs=2048), True),
    (dict(ots=64, ohs=2040), False), (dict(n=1, ots=0), True), (dict(ots=1 << 62), False),
])
def test_attention_writes_apart_from_what_steers_it(lib, kw, ok):  # noqa: F811
    a = dict(q=P, qts=512, qhs=64, hq=8, k=P, v=P, nts=128, nhs=64, layer=0, indptr=P, slots=0x50000000, bs=4, n=32, mask=P,
             words=1, scale=0.125, out=0x40000000, ots=512, ohs=64, lse=0x60000000, ws=0x80000000)
    a.update(kw)
    c = cache()
    short = lib.csgmv_tree_attention_workspace_bytes(ctypes.byref(c), 8) - 1  # refused last: nothing is launched here
    rc = lib.csgmv_tree_attention(a["q"], a["qts"], a["qhs"], a["hq"], a["k"], a["v"], a["nts"], a["nhs"], ctypes.byref(c),
                                  a["layer"], a["indptr"], a["slots"], a["bs"], a["n"], a["mask"], a["words"], a["scale"],
                                  a["out"], a["ots"], a["ohs"], a["lse"], a["ws"], short, None)
    assert rc == (CAPACITY if ok else INVALID)
    assert (b"overlap" in lib.csgmv_last_error()) is not ok


AT = {name: 0x1000000 * (i + 1) for i, name in enumerate(
    ("target", "draft", "tokens", "indptr", "first", "next", "au", "su", "path", "len", "token", "status"))}


@pytest.mark.parametrize("out,size", [("path", 4 * 2 * 5), ("len", 8), ("token", 8), ("status", 4)])
@pytest.mark.parametrize("inp,size_in", [("target", 4 * (7 * 1000 + 900)), ("draft", 4 * (7 * 904 + 900)), ("tokens", 32),
                                         ("indptr", 12), ("first", 32), ("next", 32), ("au", 32), ("su", 8)])
def test_verification_writes_apart_from_what_it_reads(lib, out, size, inp, size_in):  # noqa: F811
    """8 nodes of 2 requests, 900 tokens; the output's first and last bytes on the input's last and first."""
    for at in (AT[inp] + size_in - 4, AT[inp] - size + 4):
        a = dict(AT)
        a[out] = at
        rc = lib.csgmv_verify_drafts(a["target"], 1000, a["draft"], 904, a["tokens"], a["indptr"], a["first"], a["next"],
                                     a["au"], a["su"], 2, 8, 900, a["path"], 5, a["len"], a["token"], a["status"], None)
        assert rc == INVALID and b"overlaps" in lib.csgmv_last_error()


@pytest.mark.parametrize("name", ["page_table", "seq_lens", "page_refs", "scratch", "status"])
def test_lists_of_a_cache_call_lie_apart_from_what_its_plan_writes(lib, name):  # noqa: F811
    c = cache()
    for i, n in enumerate(("page_table", "seq_lens", "page_refs", "scratch", "status")):
        setattr(c, n, 0x1000000 * (i + 1))
    size = dict(page_table=4 * 8 * 4, seq_lens=4 * 8, page_refs=4 * 16, scratch=4 * lib.csgmv_kv_scratch_ints(16, 8), status=4)
    ref = ctypes.byref(c)
    for at in (getattr(c, name), getattr(c, name) + size[name] - 4):
        for kw in (dict(idx=at), dict(lens=at), dict(indptr=at), dict(lens=at - 12), dict(idx=at - 60)):
            assert commit(lib, c, **kw) == INVALID and b"overlaps" in lib.csgmv_last_error()
        slots = lib.csgmv_kv_commit(ref, P, P, 1 << 20, 128, 64, 32, P, 4, P, P, at, 4, None)
        assert slots == INVALID and b"overlaps" in lib.csgmv_last_error()
        for a, b in ((at, P), (P, at), (P, at - 28)):
            assert lib.csgmv_kv_fork(ref, a, b, 8, None) == INVALID and b"overlaps" in lib.csgmv_last_error()
