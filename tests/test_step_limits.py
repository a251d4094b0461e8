"""Sizes near 2^31, where a kernel's 32-bit index would run past its end: refused
before anything is launched.  CPU only: no kernel runs."""
import ctypes

import pytest

from tests.test_serving_abi import INVALID, P, UNSUPPORTED, cache, lib  # noqa: F401
from tests.test_step_abi import count, counts, process

MOST = 1 << 30


@pytest.mark.parametrize("total", [MOST + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 40])
def test_biases(lib, total):  # noqa: F811
    """The threads of a CTA begin up to 255 entries behind a list's first one, and go on in steps of 256."""
    far = 0x100000000000
    assert process(lib, bias_indptr=P, bias_tokens=far, bias_values=2 * far, bias_total=total) == INVALID
    assert b"bias_total" in lib.csgmv_last_error()


@pytest.mark.parametrize("bs", [MOST + 1, 2 ** 31 - 1])
def test_requests_of_logits(lib, bs):  # noqa: F811
    far = 0x100000000000
    assert process(lib, bs=bs, indptr=far) == UNSUPPORTED and b"bs" in lib.csgmv_last_error()


@pytest.mark.parametrize("width", [MOST + 1, 2 ** 31 - 1])
def test_accepted_paths(lib, width):  # noqa: F811
    far = 0x100000000000
    assert count(lib, counts(), idx=far, width=width, lens=P) == UNSUPPORTED and b"accept_width" in lib.csgmv_last_error()
    c = cache()
    rc = lib.csgmv_kv_commit(ctypes.byref(c), 0x10000000000, 0x20000000000, 1 << 20, 128, 64, 20, far, width, P, P + 64, None, 4, None)
    assert rc == UNSUPPORTED and b"accept_width" in lib.csgmv_last_error()
    rc = lib.csgmv_verify_drafts(0x10000000000, 1000, None, 0, *[0x1000000 * i for i in range(1, 6)], 0x6000000, 4, 20, 1000, far, width,
                                 0x7000000, 0x8000000, 0x9000000, None)
    assert rc == UNSUPPORTED and b"accept_width" in lib.csgmv_last_error()
