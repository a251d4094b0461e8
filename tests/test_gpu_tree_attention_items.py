"""Many items a CTA, one token tile each, every one of them with drafted values
that are not finite: a softmax warp that is done with an item goes on to the
next while others still end theirs, so what one item found must not be taken
for, or lost to, the next one's.

The values are exact: with K = 0 a row weighs what it sees alike, and one
infinity or NaN among what it sees decides an element whatever the rest is."""
import numpy as np
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_i32

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


# rows a kv head: 1 (half the softmax warps have none), 3, 16 (turned over); 17, 40 (quadrants without rows)
@pytest.mark.parametrize("T,group", [(1, 1), (1, 3), (2, 8), (17, 1), (5, 8)])
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float16)])
def test_items_in_succession_with_values_that_are_not_finite(T, group, d, dtype):
    bs, hkv, ps = 3000 if T == 1 else 600, 4, 16
    rng = np.random.default_rng(10 * T + group)
    lens = rng.integers(0, 17, bs)
    cache = B.KvCache.allocate(1, 1, ps, hkv, d, bs, 1, dtype=dtype)
    cache.k_pages.zero_()
    cache.v_pages.zero_()
    cache.page_table.zero_()
    cache.seq_lens.copy_(dev_i32(lens))
    n = bs * T
    q = torch.ones((n, hkv * group, d), dtype=dtype, device="cuda")
    kn = torch.zeros((n, hkv, d), dtype=dtype, device="cuda")
    vn = torch.zeros((n, hkv, d), dtype=dtype, device="cuda")
    # row t of every request: element (t + kv head) % d of what t itself holds, another value each
    kinds = torch.tensor([INF, -INF, NAN], device="cuda")
    row = torch.arange(n, device="cuda")
    for h in range(hkv):
        vn[row, h, (row % T + h) % d] = kinds[(row + h) % 3].to(dtype)
    # a row sees itself alone
    bits = dev_i32(np.tile(1 << np.arange(T, dtype=np.int64), bs).astype(np.uint32).view(np.int32).reshape(n, 1))
    indptr = dev_i32(np.arange(bs + 1) * T)
    want = vn.repeat_interleave(group, 1)
    odd = ~torch.isfinite(want)
    for _ in range(20):
        out = torch.full_like(q, 7.0)
        B.csgmv_tree_attention(q, kn, vn, cache, 0, indptr, out, mask=bits)
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        assert torch.equal(out.nan_to_num(1.0, INF, -INF)[odd], want.nan_to_num(1.0, INF, -INF)[odd])
        assert (out[~odd] == 0).all()
    assert cache.device_status() == 0
