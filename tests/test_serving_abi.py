"""Host checks of the serving operators' C calls: what they refuse before they
touch the device, and the sizes of their scratch.  CPU only: no kernel runs."""
import ctypes

import pytest

from segmented_gather_gemm_gb300 import build as sgb

OK, INVALID, CAPACITY, UNSUPPORTED = 0, -1, -2, -6
P = 0x100000  # a device pointer that is never followed


@pytest.fixture(scope="module")
def lib():
    try:
        sgb.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    from segmented_gather_gemm_gb300 import binding
    return binding.lib()


def cache(**kw):
    """4 layers of 16 pages of 16 tokens, 2 kv heads of 64, heads outside the tokens."""
    from segmented_gather_gemm_gb300 import binding
    c = binding._KvCacheC()
    for i, n in enumerate(("k_pages", "v_pages", "page_table", "seq_lens", "page_refs", "scratch", "status")):
        setattr(c, n, 0x1000 * (i + 1))
    c.layer_stride, c.page_stride, c.head_stride, c.token_stride = 16 * 2048, 2048, 1024, 64
    c.dtype, c.num_layers, c.num_pages, c.page_size = 0, 4, 16, 16
    c.num_kv_heads, c.head_dim, c.max_seqs, c.max_pages_per_seq = 2, 64, 8, 4
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_scratch_sizes(lib):
    assert lib.csgmv_kv_scratch_ints(-1, 4) == 0 and lib.csgmv_kv_scratch_ints(4, -1) == 0
    small, more, seqs = (lib.csgmv_kv_scratch_ints(*a) for a in ((16, 8), (32, 8), (16, 64)))
    assert 0 < small < more and small < seqs
    c = cache()
    assert lib.csgmv_tree_attention_workspace_bytes(None, 8) == 0
    assert lib.csgmv_tree_attention_workspace_bytes(ctypes.byref(c), 0) == 0
    d64 = lib.csgmv_tree_attention_workspace_bytes(ctypes.byref(c), 8)
    wide = cache(head_dim=128, token_stride=128, head_stride=2048, page_stride=4096)
    assert 0 < d64 < lib.csgmv_tree_attention_workspace_bytes(ctypes.byref(wide), 8)


def commit(lib, c, k=P, v=P, ls=1 << 20, ts=128, hs=64, n=32, idx=P, width=4, lens=P, indptr=P, bs=4):
    return lib.csgmv_kv_commit(None if c is None else ctypes.byref(c), k, v, ls, ts, hs, n, idx, width, lens, indptr, None,
                               bs, None)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(k_pages=None), INVALID, b"NULL"), (dict(status=None), INVALID, b"NULL"),
    (dict(k_pages=0x1008), INVALID, b"16-byte"), (dict(seq_lens=0x1002), INVALID, b"4-byte"),
    (dict(dtype=1), INVALID, b"dtype"), (dict(num_layers=0), INVALID, b"positive"),
    (dict(num_pages=0), INVALID, b"positive"), (dict(max_seqs=-3), INVALID, b"positive"),
    (dict(num_layers=20000), UNSUPPORTED, b"layers"), (dict(page_size=12), UNSUPPORTED, b"page_size"),
    (dict(page_size=4), UNSUPPORTED, b"page_size"), (dict(page_size=8192), UNSUPPORTED, b"page_size"),
    (dict(num_pages=1 << 25), UNSUPPORTED, b"pages"), (dict(max_seqs=1 << 21), UNSUPPORTED, b"sequences"),
    (dict(max_pages_per_seq=1 << 28), UNSUPPORTED, b"tokens"), (dict(head_dim=60), UNSUPPORTED, b"head_dim"),
    (dict(head_dim=2048), UNSUPPORTED, b"head_dim"), (dict(num_kv_heads=2000), UNSUPPORTED, b"kv heads"),
    (dict(token_stride=60), INVALID, b"strides"), (dict(layer_stride=-8), INVALID, b"strides"),
    (dict(page_stride=1 << 32), UNSUPPORTED, b"page_stride"), (dict(head_stride=512), INVALID, b"overlap"),
    (dict(token_stride=56), INVALID, b"overlap"), (dict(page_stride=1024), INVALID, b"overlap")])
def test_caches_that_are_refused(lib, kw, rc, msg):
    c = cache(**kw)
    ref = ctypes.byref(c)
    for call in (lambda: commit(lib, c), lambda: lib.csgmv_kv_fork(ref, P, P, 1, None),
                 lambda: lib.csgmv_kv_free(ref, P, None, 1, None), lambda: lib.csgmv_kv_compact(ref, None),
                 lambda: lib.csgmv_kv_copy_pages(ref, P, P, 1, None), lambda: attend(lib, c)):
        assert call() == rc
        assert msg in lib.csgmv_last_error()


def test_cache_calls_that_are_refused(lib):
    c = cache()
    ref = ctypes.byref(c)
    assert commit(lib, None) == INVALID
    assert commit(lib, c, bs=-1) == INVALID and commit(lib, c, n=-1) == INVALID
    assert commit(lib, c, bs=9) == CAPACITY and b"max_seqs" in lib.csgmv_last_error()
    assert commit(lib, c, n=1 << 31) == UNSUPPORTED
    assert commit(lib, c, lens=None) == INVALID and commit(lib, c, indptr=None) == INVALID
    assert commit(lib, c, width=0) == INVALID and b"accept_width" in lib.csgmv_last_error()
    assert commit(lib, c, k=None) == INVALID and commit(lib, c, v=P + 8) == INVALID
    assert commit(lib, c, ts=100) == INVALID and commit(lib, c, hs=0) == INVALID and commit(lib, c, ls=4) == INVALID
    # nothing to do is no error, whatever else is missing
    assert commit(lib, c, bs=0, lens=None) == OK and commit(lib, c, n=0, k=None) == OK
    for call in (lib.csgmv_kv_fork, lib.csgmv_kv_free):
        assert call(ref, P, P, -1, None) == INVALID and call(ref, P, P, 9, None) == CAPACITY
        assert call(ref, None, P, 1, None) == INVALID and call(ref, None, None, 0, None) == OK
    assert lib.csgmv_kv_fork(ref, P, None, 1, None) == INVALID
    assert lib.csgmv_kv_copy_pages(ref, P, P, -1, None) == INVALID
    assert lib.csgmv_kv_copy_pages(ref, P, None, 1, None) == INVALID
    assert lib.csgmv_kv_copy_pages(ref, None, None, 0, None) == OK


def attend(lib, c, q=P, hq=8, qts=512, qhs=64, k=P, v=P, nts=128, nhs=64, layer=0, indptr=P, bs=4, n=32, mask=P, words=1,
           scale=0.125, out=0x40000000, ots=512, ohs=64, lse=None, ws=0x80000000, wsb=1 << 30):
    return lib.csgmv_tree_attention(q, qts, qhs, hq, k, v, nts, nhs, None if c is None else ctypes.byref(c), layer, indptr,
                                    None, bs, n, mask, words, scale, out, ots, ohs, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(hq=0), INVALID, b"num_q_heads"), (dict(hq=7), INVALID, b"num_q_heads"), (dict(hq=260), UNSUPPORTED, b"128"),
    (dict(layer=4), INVALID, b"layer"), (dict(layer=-1), INVALID, b"layer"), (dict(bs=-1), INVALID, b"negative"),
    (dict(n=1 << 25), UNSUPPORTED, b"2^24"), (dict(bs=16001), UNSUPPORTED, b"16000"), (dict(q=None), INVALID, b"NULL"),
    (dict(out=None), INVALID, b"NULL"), (dict(indptr=None), INVALID, b"NULL"), (dict(q=P + 4), INVALID, b"16-byte"),
    (dict(qts=500), INVALID, b"strides"), (dict(ohs=-64), INVALID, b"strides"), (dict(k=None), INVALID, b"k_new"),
    (dict(nts=0), INVALID, b"k_new"), (dict(words=0), INVALID, b"mask_words"), (dict(lse=P + 2), INVALID, b"lse"),
    (dict(scale=0.0), INVALID, b"scale"), (dict(scale=float("nan")), INVALID, b"scale"),
    (dict(scale=float("inf")), INVALID, b"scale"), (dict(ws=None), INVALID, b"workspace"),
    (dict(ws=0x80000008), INVALID, b"workspace"), (dict(wsb=1024), CAPACITY, b"needed"),
    (dict(out=0x3000), INVALID, b"overlaps"), (dict(lse=0x4000), INVALID, b"overlaps"),
    (dict(ws=0x40000000), INVALID, b"overlaps"), (dict(out=0x7000 - 64), INVALID, b"overlaps")])
def test_attention_calls_that_are_refused(lib, kw, rc, msg):
    assert attend(lib, cache(), **kw) == rc
    assert msg in lib.csgmv_last_error()


def test_attention_without_work(lib):
    assert attend(lib, None) == INVALID
    assert attend(lib, cache(), bs=0, q=None) == OK and attend(lib, cache(), n=0, out=None) == OK
    assert attend(lib, cache(head_dim=32)) == UNSUPPORTED and b"head_dim" in lib.csgmv_last_error()


def test_tree_calls_that_are_refused(lib):
    def build(parents=P, indptr=P, bs=2, n=8, words=1, mask=P, status=P):
        return lib.csgmv_build_draft_tree(parents, indptr, bs, n, words, mask, P, P, P, status, None)

    assert build(bs=-1) == INVALID and build(n=-1) == INVALID and build(n=1 << 31) == UNSUPPORTED
    assert build(words=0) == UNSUPPORTED and build(words=9) == UNSUPPORTED
    assert build(parents=None) == INVALID and build(mask=None) == INVALID and build(status=None) == INVALID
    assert build(bs=0, mask=None) == OK and build(n=0, parents=None) == OK


def test_verify_calls_that_are_refused(lib):
    def verify(t=P, ts=1000, d=None, ds=0, tokens=P, indptr=P, u=P, bs=2, n=8, vocab=1000, path=P, width=4, status=P):
        return lib.csgmv_verify_drafts(t, ts, d, ds, tokens, indptr, P, P, u, P, bs, n, vocab, path, width, P, P, status, None)

    assert verify(bs=-1) == INVALID and verify(n=-1) == INVALID and verify(n=1 << 31) == UNSUPPORTED
    assert verify(vocab=0) == UNSUPPORTED and verify(vocab=(1 << 18) + 1) == UNSUPPORTED
    assert verify(width=0) == INVALID and b"accept_width" in lib.csgmv_last_error()
    assert verify(ts=999) == INVALID and b"vocab_size" in lib.csgmv_last_error()
    assert verify(d=P, ds=999) == INVALID and verify(d=P + 2, ds=1000) == INVALID and verify(t=P + 1) == INVALID
    for kw in (dict(t=None), dict(tokens=None), dict(indptr=None), dict(u=None), dict(path=None), dict(status=None)):
        assert verify(**kw) == INVALID and b"NULL" in lib.csgmv_last_error()
    assert verify(bs=0, indptr=None) == OK
