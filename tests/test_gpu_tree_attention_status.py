"""After a wait inside the attention kernel ran out, its waits are no longer sat
out: the calls that follow must do nothing until the status bit is cleared,
instead of running without them.  (The bit is set from the host here.)"""
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_i32

pytestmark = pytest.mark.gpu

TIMEOUT = 1 << 30


@pytest.mark.parametrize("T,L", [([1, 3, 0], [40, 0, 7]), ([200, 33], [300, 5000]), ([1] * 500, [20] * 500)])
def test_calls_after_a_wait_that_ran_out_give_no_output(T, L):
    pages = 8
    g = torch.Generator(device="cuda")
    g.manual_seed(len(T))

    def draw(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    cache = B.KvCache(draw(1, pages, 2, 16, 64), draw(1, pages, 2, 16, 64),
                      (torch.arange(len(T) * 320, dtype=torch.int32, device="cuda") % pages).view(len(T), 320),
                      dev_i32(L), torch.ones(pages, dtype=torch.int32, device="cuda"))
    n = sum(T)
    q, kn, vn = draw(n, 8, 64), draw(n, 2, 64), draw(n, 2, 64)
    ptr = dev_i32([sum(T[:i]) for i in range(len(T) + 1)])

    def call():
        out, lse = torch.full_like(q, 7.0), torch.full((n, 8), 7.0, device="cuda")
        B.csgmv_tree_attention(q, kn, vn, cache, 0, ptr, out, lse=lse)
        return out, lse

    want = call()
    assert cache.device_status() == 0 and torch.isfinite(want[0]).all() and not (want[1] == 7).any()
    cache.status.fill_(TIMEOUT)
    for _ in range(3):
        out, lse = call()
        assert (out == 7).all() and (lse == 7).all()
    assert cache.device_status() == TIMEOUT
    cache.status.zero_()
    out, lse = call()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and cache.device_status() == 0
