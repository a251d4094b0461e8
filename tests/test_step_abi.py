"""Host checks of the calls between the projections, the attention and the
verification: what they refuse before they touch the device.  CPU only: no
kernel runs."""
import ctypes

import pytest

from tests.test_serving_abi import CAPACITY, INVALID, OK, P, UNSUPPORTED, cache, lib  # noqa: F401

NAN, INF = float("nan"), float("inf")


def norm(kind=1, w=P, b=None, eps=1e-6):
    from segmented_gather_gemm_gb300 import binding
    return ctypes.byref(binding._NormC(w, b, eps, kind))


def add_norm(lib, x=0x10000000, xs=512, dtype=0, r=0x20000000, rs=512, rtype=0, gate=None, gs=0, post=None, pre="rms", scale=1.0,
             n=64, hidden=512, ro=0x30000000, ros=512, out=0x40000000, os=512):
    return lib.csgmv_add_norm(x, xs, dtype, r, rs, rtype, gate, gs, post, norm() if pre == "rms" else pre, scale, n, hidden, ro,
                              ros, out, os, None)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(dtype=3), INVALID, b"dtype"), (dict(rtype=2), INVALID, b"dtype"), (dict(dtype=1, rtype=0), INVALID, b"dtype"),
    (dict(n=-1), INVALID, b"negative"), (dict(n=1 << 31), UNSUPPORTED, b"int32"), (dict(hidden=0), UNSUPPORTED, b"hidden"),
    (dict(hidden=16385), UNSUPPORTED, b"hidden"), (dict(pre=3), INVALID, b"kind"), (dict(scale=NAN), INVALID, b"finite"),
    (dict(scale=INF), INVALID, b"finite"), (dict(x=None), INVALID, b"NULL"), (dict(out=None, ro=None), INVALID, b"NULL"),
    (dict(out=None), INVALID, b"without out"), (dict(x=0x10000001), INVALID, b"aligned"), (dict(rtype=1, r=0x20000002), INVALID, b"aligned"),
    (dict(xs=-512), INVALID, b"stride"), (dict(gs=1 << 41, gate=P), INVALID, b"stride"), (dict(os=511), INVALID, b"overlap"),
    (dict(ros=0), INVALID, b"overlap"),
    # outputs over inputs, weights and each other
    (dict(out=0x10000002), INVALID, b"an input"), (dict(ro=0x10000000, ros=520), INVALID, b"an input"),
    (dict(out=0x20000000, rtype=1), INVALID, b"an input"), (dict(out=0x40000000, gate=0x40000000, gs=0), INVALID, b"an input"),
    (dict(out=P - 16), INVALID, b"weight"), (dict(ro=P + 512), INVALID, b"weight"), (dict(out=0x30000200), INVALID, b"each other"),
])
def test_add_norm_calls_that_are_refused(lib, kw, rc, msg):  # noqa: F811
    if isinstance(kw.get("pre"), int):
        kw = dict(kw, pre=norm(kind=kw["pre"]))
    assert add_norm(lib, **kw) == rc
    assert msg in lib.csgmv_last_error()


def test_norms_that_are_refused(lib):  # noqa: F811
    for bad, msg in ((norm(eps=-1.0), b"eps"), (norm(eps=NAN), b"eps"), (norm(eps=INF), b"eps"), (norm(w=P + 1), b"aligned"),
                     (norm(b=P + 1), b"aligned"), (norm(kind=-1), b"kind")):
        assert add_norm(lib, pre=bad) == INVALID and msg in lib.csgmv_last_error()
        assert add_norm(lib, post=bad) == INVALID and msg in lib.csgmv_last_error()


def test_add_norm_of_nothing(lib):  # noqa: F811
    assert add_norm(lib, n=0, x=None, out=None) == OK


def rope(turns=P, scale=1.0, rot=64, il=0):
    from segmented_gather_gemm_gb300 import binding
    return ctypes.byref(binding._RopeC(turns, scale, rot, il))


Q, K, V, QO, KO, POS, SLOTS = (0x10000000 * i for i in range(1, 8))


def rotary(lib, r="rope", dtype=0, d=64, pos=POS, n=32, q=Q, qts=512, qhs=64, hq=8, k=K, kts=128, khs=64, hk=2, qo=QO, qots=512,
           qohs=64, ko=KO, kots=128, kohs=64, inverse=0):
    return lib.csgmv_rotary(rope() if r == "rope" else r, dtype, d, pos, n, q, qts, qhs, hq, k, kts, khs, hk, qo, qots, qohs, ko,
                            kots, kohs, inverse, None)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(r=None), INVALID, b"rope"), (dict(dtype=3), INVALID, b"dtype"), (dict(d=0), UNSUPPORTED, b"head_dim"),
    (dict(d=1025), UNSUPPORTED, b"head_dim"), (dict(d=60), INVALID, b"rotary_dim"), (dict(n=-1), INVALID, b"negative"),
    (dict(n=1 << 31), UNSUPPORTED, b"int32"), (dict(inverse=2), INVALID, b"inverse"), (dict(hq=-1), UNSUPPORTED, b"heads"),
    (dict(hk=5000), UNSUPPORTED, b"heads"), (dict(q=None), INVALID, b"NULL"), (dict(ko=None), INVALID, b"NULL"),
    (dict(q=Q + 1), INVALID, b"aligned"), (dict(qts=-512), INVALID, b"stride"), (dict(kohs=1 << 41), INVALID, b"stride"),
    (dict(qohs=63), INVALID, b"overlap"), (dict(kots=64), INVALID, b"overlap"), (dict(pos=None), INVALID, b"positions"),
    (dict(pos=POS + 2), INVALID, b"positions"), (dict(qo=Q, qots=1024), INVALID, b"an output"), (dict(qo=Q + 2), INVALID, b"an output"),
    (dict(qo=K), INVALID, b"an output"), (dict(ko=Q), INVALID, b"an output"), (dict(ko=QO + 256), INVALID, b"an output"),
    (dict(qo=POS - 64), INVALID, b"an output"), (dict(qo=P), INVALID, b"an output"),
    # slices of one tensor that run into each other
    (dict(q=Q, qts=640, k=Q + 1024 - 2, kts=640, qo=Q, qots=640), INVALID, b"an output")])
def test_rotary_calls_that_are_refused(lib, kw, rc, msg):  # noqa: F811
    assert rotary(lib, **kw) == rc
    assert msg in lib.csgmv_last_error()


def test_ropes_that_are_refused(lib):  # noqa: F811
    for bad, msg in ((rope(rot=-2), b"rotary_dim"), (rope(rot=63), b"rotary_dim"), (rope(rot=66), b"rotary_dim"),
                     (rope(turns=None), b"turns"), (rope(turns=P + 4), b"turns"), (rope(il=2), b"interleaved"),
                     (rope(scale=NAN), b"scale"), (rope(scale=INF), b"scale")):
        assert rotary(lib, r=bad) == INVALID and msg in lib.csgmv_last_error()
        assert append(lib, cache(), r=bad) == INVALID and msg in lib.csgmv_last_error()


def test_rotary_of_nothing(lib):  # noqa: F811
    assert rotary(lib, n=0, q=None, pos=None) == OK
    assert rotary(lib, hq=0, hk=0, q=None, k=None, pos=None) == OK


@pytest.mark.parametrize("freq,want", [(0.0, 0), (2 * 3.141592653589793, 0), (3.141592653589793, 1 << 63),
                                       (-3.141592653589793 / 2, 3 << 62), (-1e-30, 0), (3.141592653589793 * 2 ** -40, 1 << 23)])
def test_turns(lib, freq, want):  # noqa: F811
    """Whole turns are none, negative ones count from behind."""
    out = (ctypes.c_uint64 * 1)(7)
    assert lib.csgmv_rope_turns((ctypes.c_double * 1)(freq), 1, out) == OK
    assert out[0] == want


def test_turns_that_are_refused(lib):  # noqa: F811
    two = (ctypes.c_double * 2)(1.0, INF)
    out = (ctypes.c_uint64 * 2)(7, 7)
    assert lib.csgmv_rope_turns(two, 2, out) == INVALID and list(out) == [7, 7]
    assert lib.csgmv_rope_turns(two, -1, out) == INVALID and lib.csgmv_rope_turns(None, 1, out) == INVALID
    assert lib.csgmv_rope_turns(None, 0, None) == OK


def test_frequencies():
    """Scaled positions, by what they promise: factors at both ends, the blend in between."""
    import torch

    from segmented_gather_gemm_gb300 import binding as B
    f, one = B.rope_frequencies(64, 10000.0)
    assert one == 1.0 and f[0] == 1.0 and abs(float(f[16]) - 0.01) < 1e-15
    assert torch.equal(B.rope_frequencies(64, 10000.0, ("linear", 4.0))[0] * 4, f)
    g, one = B.rope_frequencies(64, 10000.0, ("ntk", 4.0))
    assert one == 1.0 and g[0] == 1.0 and abs(float(g[-1] * 4 / f[-1]) - 1) < 1e-12
    g, one = B.rope_frequencies(64, 10000.0, ("wavelength", 8.0, 1.0, 4.0, 8192.0))
    turns = 8192 * f / (2 * 3.141592653589793)
    assert one == 1.0 and torch.equal(g[turns >= 4], f[turns >= 4]) and torch.allclose(g[turns <= 1] * 8, f[turns <= 1], rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and bool(((g < f) & (g > f / 8))[mid].all())
    g, scale = B.rope_frequencies(64, 10000.0, ("yarn", 4.0, 8192))
    assert abs(scale - 1.1386294361119891) < 1e-12
    assert torch.equal(g[turns > 40], f[turns > 40]) and torch.allclose(g[turns < 0.7] * 4, f[turns < 0.7], rtol=1e-14)
    for bad in (("linear",), ("linear", 0.0), ("other", 1.0), ("wavelength", 8.0, 4.0, 1.0, 8192.0), ("yarn", 4.0)):
        with pytest.raises(B.CsgmvError):
            B.rope_frequencies(64, 10000.0, bad)
    with pytest.raises(B.CsgmvError):
        B.rope_frequencies(63)


def extend(lib, c, lens=0x10000, indptr=0x20000, seqs=0x30000, bs=4, n=32, slots=0x40000, pos=0x50000, before=0x60000):
    return lib.csgmv_kv_extend(None if c is None else ctypes.byref(c), lens, indptr, seqs, bs, n, slots, pos, before, None)


def far(**kw):
    """A cache whose pages and scratch are away from the small addresses."""
    return cache(k_pages=0x100000000, v_pages=0x200000000, **kw)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(bs=-1), INVALID, b"negative"), (dict(n=-1), INVALID, b"negative"), (dict(bs=9), CAPACITY, b"max_seqs"),
    (dict(n=1 << 31), UNSUPPORTED, b"int32"), (dict(indptr=None), INVALID, b"tree_indptr"), (dict(slots=None), INVALID, b"NULL"),
    (dict(pos=None), INVALID, b"NULL"), (dict(slots=0x40004), INVALID, b"aligned"), (dict(lens=0x10002), INVALID, b"aligned"),
    # over one another, the cache's bookkeeping, its scratch, its pages
    (dict(pos=0x40000), INVALID, b"overlaps"), (dict(before=0x50000), INVALID, b"overlaps"), (dict(lens=0x40000), INVALID, b"overlaps"),
    (dict(indptr=0x60000), INVALID, b"overlaps"), (dict(seqs=0x50008), INVALID, b"overlaps"), (dict(before=0x4000), INVALID, b"overlaps"),
    (dict(before=0x5000), INVALID, b"overlaps"), (dict(slots=0x3000), INVALID, b"overlaps"), (dict(pos=0x6000), INVALID, b"overlaps"),
    (dict(lens=0x6000), INVALID, b"overlaps"), (dict(pos=0x100000100), INVALID, b"overlaps"), (dict(slots=0x200000000), INVALID, b"overlaps")])
def test_extend_calls_that_are_refused(lib, kw, rc, msg):  # noqa: F811
    assert extend(lib, far(), **kw) == rc
    assert msg in lib.csgmv_last_error()


def test_extend_of_nothing(lib):  # noqa: F811
    assert extend(lib, None) == INVALID
    assert extend(lib, far(), bs=0, n=0, indptr=None, slots=None, pos=None, before=None) == OK


def append(lib, c, layer=1, r="rope", pos=POS, slots=SLOTS, n=32, q=Q, qts=512, qhs=64, hq=8, k=K, kts=128, khs=64, v=V, vts=128,
           vhs=64, qo=QO, qots=512, qohs=64, ko=None, kots=128, kohs=64):
    return lib.csgmv_kv_append(None if c is None else ctypes.byref(c), layer, rope() if r == "rope" else r, pos, slots, n, q, qts,
                               qhs, hq, k, kts, khs, v, vts, vhs, qo, qots, qohs, ko, kots, kohs, None)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(layer=4), INVALID, b"layer"), (dict(layer=-1), INVALID, b"layer"), (dict(n=-1), INVALID, b"negative"),
    (dict(n=1 << 31), UNSUPPORTED, b"int32"), (dict(hq=-1), UNSUPPORTED, b"heads"), (dict(q=None), INVALID, b"NULL"),
    (dict(qo=None), INVALID, b"NULL"), (dict(k=None), INVALID, b"NULL"), (dict(v=None), INVALID, b"NULL"),
    (dict(v=V + 1), INVALID, b"aligned"), (dict(kts=-8), INVALID, b"stride"), (dict(qohs=0), INVALID, b"overlap"),
    (dict(slots=None), INVALID, b"slots"), (dict(slots=SLOTS + 4), INVALID, b"slots"), (dict(pos=None), INVALID, b"positions"),
    (dict(qo=K), INVALID, b"an output"), (dict(qo=V), INVALID, b"an output"), (dict(ko=V), INVALID, b"an output"),
    (dict(ko=Q), INVALID, b"an output"), (dict(ko=QO), INVALID, b"an output"), (dict(ko=K, kots=256), INVALID, b"an output"),
    (dict(qo=SLOTS), INVALID, b"an output"), (dict(ko=POS), INVALID, b"an output"), (dict(qo=P - 64), INVALID, b"an output"),
    # the cache's pages and bookkeeping
    (dict(qo=0x100000000), INVALID, b"an output"), (dict(ko=0x200000100), INVALID, b"an output"), (dict(k=0x100000000), INVALID, b"an output"),
    (dict(v=0x200000000), INVALID, b"an output"), (dict(slots=0x100000000), INVALID, b"an output"), (dict(qo=0x3000), INVALID, b"an output")])
def test_append_calls_that_are_refused(lib, kw, rc, msg):  # noqa: F811
    assert append(lib, far(), **kw) == rc
    assert msg in lib.csgmv_last_error()


def test_append_of_nothing(lib):  # noqa: F811
    assert append(lib, None) == INVALID
    assert append(lib, far(), n=0, k=None, slots=None) == OK


def counts(**kw):
    from segmented_gather_gemm_gb300 import binding
    c = binding._TokenCountsC(0x1000000, 0x2000000, 0x3000000, 0x3100000, 8, 1000)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def count(lib, c, tokens=0x5000000, n=50, indptr=0x5100000, idx=None, width=0, lens=None, seqs=None, bs=4, prompt=0):
    return lib.csgmv_count_tokens(None if c is None else ctypes.byref(c), tokens, n, indptr, idx, width, lens, seqs, bs, prompt, None)


BAD_COUNTS = [(dict(counts=None), INVALID, b"NULL"), (dict(status=0x3100002), INVALID, b"aligned"), (dict(max_seqs=0), INVALID, b"positive"),
              (dict(vocab_size=-1), INVALID, b"positive"), (dict(vocab_size=(1 << 18) + 1), UNSUPPORTED, b"2^18"),
              (dict(max_seqs=(1 << 20) + 1), UNSUPPORTED, b"2^20"), (dict(seen=0x1000010), INVALID, b"overlap"),
              (dict(num_seen=0x1000000 + 31996), INVALID, b"overlap"), (dict(status=0x3000004), INVALID, b"overlap")]


@pytest.mark.parametrize("kw,rc,msg", BAD_COUNTS)
def test_counts_that_are_refused(lib, kw, rc, msg):  # noqa: F811
    c = counts(**kw)
    for call in (lambda: count(lib, c), lambda: lib.csgmv_count_reset(ctypes.byref(c), P, 1, None),
                 lambda: lib.csgmv_count_fork(ctypes.byref(c), P, P + 64, 1, None), lambda: process(lib, counts=c)):
        assert call() == rc and msg in lib.csgmv_last_error()


@pytest.mark.parametrize("kw,msg", [
    (dict(bs=-1), b"negative"), (dict(n=-1), b"negative"), (dict(prompt=2), b"prompt"), (dict(tokens=None), b"NULL"),
    (dict(indptr=None), b"NULL"), (dict(idx=P, width=0, lens=P), b"accept_index"), (dict(idx=P, width=4), b"accept_index"),
    (dict(tokens=0x5000002), b"aligned"), (dict(tokens=0x1000000), b"overlaps"), (dict(seqs=0x3000000), b"overlaps"),
    (dict(lens=0x3100000), b"overlaps"), (dict(idx=0x2000000, width=4, lens=P), b"overlaps")])
def test_count_calls_that_are_refused(lib, kw, msg):  # noqa: F811
    assert count(lib, counts(), **kw) == INVALID and msg in lib.csgmv_last_error()


def test_other_count_calls_that_are_refused(lib):  # noqa: F811
    c = ctypes.byref(counts())
    assert count(lib, None) == INVALID and count(lib, counts(), n=1 << 31) == UNSUPPORTED
    assert lib.csgmv_count_reset(c, P, -1, None) == INVALID and lib.csgmv_count_reset(c, None, 1, None) == INVALID
    assert lib.csgmv_count_reset(c, 0x1000000, 1, None) == INVALID and lib.csgmv_count_reset(None, P, 1, None) == INVALID
    assert lib.csgmv_count_fork(c, P, P, -1, None) == INVALID and lib.csgmv_count_fork(c, P, P, 9, None) == CAPACITY
    assert lib.csgmv_count_fork(c, P, None, 1, None) == INVALID and lib.csgmv_count_fork(c, 0x3000000, P, 1, None) == INVALID
    # nothing to do
    assert count(lib, counts(), bs=0, tokens=None) == OK and count(lib, counts(), n=0, tokens=None) == OK
    assert lib.csgmv_count_reset(c, None, 0, None) == OK and lib.csgmv_count_fork(c, None, None, 0, None) == OK


def process(lib, counts=None, rules=True, logits=0x40000000, dtype=0, ls=1000, indptr=0x5000000, seqs=None, bs=4, n=20, vocab=1000,
            drafts=None, mask=None, words=1, softmax=1, out=0x50000000, os=1000, status=0x6000000, **kw):
    from segmented_gather_gemm_gb300 import binding
    r = binding._LogitRulesC()
    if counts is not None:
        r.counts = ctypes.pointer(counts)
    r.status = status
    for k, v in kw.items():
        setattr(r, k, v)
    return lib.csgmv_process_logits(logits, dtype, ls, indptr, seqs, bs, n, vocab, ctypes.byref(r) if rules else None, drafts, mask,
                                    words, softmax, out, os, None)


@pytest.mark.parametrize("kw,rc,msg", [
    (dict(dtype=3), INVALID, b"dtype"), (dict(bs=-1), INVALID, b"negative"), (dict(n=-1), INVALID, b"negative"),
    (dict(n=1 << 24), UNSUPPORTED, b"2^24"), (dict(vocab=0), UNSUPPORTED, b"vocab"), (dict(vocab=(1 << 18) + 1), UNSUPPORTED, b"vocab"),
    (dict(rules=False), INVALID, b"rules"), (dict(status=None), INVALID, b"status"), (dict(status=0x6000002), INVALID, b"status"),
    (dict(bias_total=-1), INVALID, b"bias_total"), (dict(bias_indptr=P, bias_total=4), INVALID, b"bias_tokens"),
    (dict(num_allow=-1), INVALID, b"num_allow"), (dict(allow_index=P, num_allow=1), INVALID, b"allow is NULL"),
    (dict(allow_index=P, allow=P + 4096, num_allow=1, allow_words=31), INVALID, b"allow_words"), (dict(softmax=2), INVALID, b"softmax"),
    (dict(drafts=P, mask=P + 4096, words=9), UNSUPPORTED, b"mask_words"), (dict(drafts=P, mask=P + 4096, words=0), UNSUPPORTED, b"mask_words"),
    (dict(logits=None), INVALID, b"NULL"), (dict(out=None), INVALID, b"NULL"), (dict(indptr=None), INVALID, b"NULL"),
    (dict(logits=0x40000001), INVALID, b"aligned"), (dict(out=0x50000002), INVALID, b"aligned"), (dict(ls=-1), INVALID, b"stride"),
    (dict(os=999), INVALID, b"overlap"), (dict(os=1 << 41), INVALID, b"stride"),
    # out over what is read
    (dict(out=0x40000000), INVALID, b"overlaps logits"), (dict(out=0x40000000, dtype=1, os=1004), INVALID, b"overlaps logits"),
    (dict(indptr=0x50000000), INVALID, b"overlaps"), (dict(temperature=0x50000100), INVALID, b"overlaps"),
    (dict(seqs=0x50000100), INVALID, b"overlaps"), (dict(repetition=0x50000002), INVALID, b"aligned"),
    (dict(drafts=0x50000100, mask=P), INVALID, b"overlaps"), (dict(drafts=P, mask=0x50000100), INVALID, b"overlaps"),
    (dict(allow_index=P, allow=0x50000000, num_allow=1, allow_words=32), INVALID, b"overlaps"), (dict(status=0x50000000), INVALID, b"status"),
    (dict(status=0x40000000), INVALID, b"status"), (dict(indptr=0x6000000), INVALID, b"status")])
def test_process_calls_that_are_refused(lib, kw, rc, msg):  # noqa: F811
    assert process(lib, **kw) == rc and msg in lib.csgmv_last_error()


def test_process_with_counts_that_do_not_fit(lib):  # noqa: F811
    assert process(lib, counts=counts(vocab_size=999)) == INVALID and b"999" in lib.csgmv_last_error()
    assert process(lib, counts=counts(), out=0x1000000) == INVALID and b"counts" in lib.csgmv_last_error()
    assert process(lib, counts=counts(), status=0x1000000) == INVALID and b"status" in lib.csgmv_last_error()
    assert process(lib, bs=0, logits=None) == OK and process(lib, n=0, logits=None) == OK
