"""Host checks of the serving operators' C calls that keep sizes within what the
kernels' arithmetic holds, and buffers that steer a kernel apart from what it
writes.  CPU only: no kernel runs."""
import pytest

from tests.test_serving_abi import INVALID, P, UNSUPPORTED, attend, cache, lib  # noqa: F401


def test_rows_of_a_kv_head_fit_30_bits(lib):  # noqa: F811
    most = (1 << 24) - 1
    for n, hq in ((most, 256), (1 << 23, 258 // 2 * 2), (most, 2 * 65)):  # 128, 129 and 65 query heads a kv head
        assert attend(lib, cache(), n=n, hq=hq) == UNSUPPORTED
    assert attend(lib, cache(), n=most, hq=2 * 65) == UNSUPPORTED and b"2^30" in lib.csgmv_last_error()
    # 64 of them fit: refused for the next thing that is wrong
    assert attend(lib, cache(), n=most, hq=2 * 64, q=None) == INVALID and b"NULL" in lib.csgmv_last_error()
