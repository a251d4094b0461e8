"""Batches whose estimated cost, by which the axis is cut, does not fit 32 bits:
a prompt that has to be right, and one that is refused.

Tolerance: as for shorter rows (u = 2^-9, the weights' and the output's
rounding; a score's and an exponential's errors), and for sums of n terms in
fp32: O grows in chains of n / 16 products, cut and not rounded at worst (n / 16
steps of 2^-23), a row's sum in chains of n / 4 (steps of 2^-24)."""
import numpy as np
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_i32

pytestmark = pytest.mark.gpu


def test_a_prompt_beyond_32_bits_of_cost():
    """110000 rows of 128 query heads on one kv head: 2.5e9 units, between
    two small requests that share the axis with it."""
    T, L, hq, d, ps = [3, 110000, 5], [100, 0, 40], 128, 64, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def draw(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    n = sum(T)
    cache = B.KvCache(draw(1, 16, 1, ps, d), draw(1, 16, 1, ps, d),
                      dev_i32(np.arange(21).reshape(3, 7) % 16), dev_i32(L), torch.ones(16, dtype=torch.int32, device="cuda"))
    q, kn, vn = draw(n, hq, d, std=2.0), draw(n, 1, d), draw(n, 1, d)
    out = torch.full_like(q, 7.0)
    lse = torch.full((n, hq), 7.0, device="cuda")
    ptr = np.concatenate([[0], np.cumsum(T)])
    B.csgmv_tree_attention(q, kn, vn, cache, 0, dev_i32(ptr), out, lse=lse)
    assert cache.device_status() == 0
    assert torch.isfinite(lse).all() and torch.isfinite(out).all()
    u = 2.0 ** -9
    for b in range(3):
        pages = (torch.arange(7) + 7 * b) % 16
        kc, vc = (pool[0, pages, 0].reshape(-1, d)[:L[b]] for pool in (cache.k_pages, cache.v_pages))
        rows = range(T[b]) if T[b] < 10 else (0, 1, 126, 127, 128, 31007, 54999, 77777, 109998, 109999)
        for t in rows:
            at = int(ptr[b]) + t
            k = torch.cat([kc, kn[ptr[b]:at + 1, 0]]).double()
            v = torch.cat([vc, vn[ptr[b]:at + 1, 0]]).double()
            a = q[at].double() @ k.T * d ** -0.5
            w = torch.softmax(a, 1)
            ref, absum, rl = w @ v, w @ v.abs(), torch.logsumexp(a, 1)
            big = float((q[at].double().abs() @ k.abs().T).max()) * d ** -0.5
            m = k.shape[0]
            off = (d + 16) * 2.0 ** -24 * big + 2.0 ** -18
            tol = (u * 1.01 + 2 * off + m / 16 * 2.0 ** -23) * absum + (u * 1.01 + m / 4 * 2.0 ** -24) * ref.abs()
            err = (out[at].double() - ref).abs()
            assert (err <= tol).all(), (b, t, float((err - tol).max()))
            le = (lse[at].double() - rl).abs()
            assert (le <= off + m / 4 * 2.0 ** -24 + 2.0 ** -22 * rl.abs()).all(), (b, t, float(le.max()))


def test_more_than_the_cut_can_count_is_refused_as_a_whole():
    """16384 rows of 128 query heads over 2^30 - 4096 cached tokens, all in one
    page: 3.6e12 units, 1.8e12 with two CTAs a part, both past 2^40."""
    d, ps, pages = 64, 4096, (1 << 18) - 1
    table = torch.zeros((2, pages), dtype=torch.int32, device="cuda")
    zero = torch.zeros((1, 1, 1, ps, d), dtype=torch.bfloat16, device="cuda")
    cache = B.KvCache(zero, zero.clone(), table, dev_i32([ps * pages, 40]), torch.ones(1, dtype=torch.int32, device="cuda"))
    n = 16384
    q = torch.zeros((n + 1, 128, d), dtype=torch.bfloat16, device="cuda")
    kn = torch.zeros((n + 1, 1, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((n + 1, 128), 7.0, device="cuda")
    B.csgmv_tree_attention(q, kn, kn, cache, 0, dev_i32([0, n, n + 1]), out, lse=lse)
    assert cache.device_status() == 4
    assert (out == 7).all() and (lse == 7).all()
    # the same cache, without the one that is too much
    cache.status.zero_()
    B.csgmv_tree_attention(q[n:], kn[n:], kn[n:], cache, 0, dev_i32([0, 1]), out[n:], seq_slots=dev_i32([1]), lse=lse[n:])
    assert cache.device_status() == 0
    assert (out[n:] == 0).all() and torch.allclose(lse[n], torch.full((128,), 41.0, device="cuda").log(), rtol=0, atol=1e-5)
