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
