"""How many bits of the softmax weights meet V.

Scores are exact (one element of Q and of K is not zero, both short numbers, and
the scale is a power of two) and tokens come in pairs of nearly the same weight
with V of opposite signs, so that an output is far smaller than the sum of its
terms and its own rounding cannot hide the weights'.

Tolerance, relative to sum w |v|: the weights' rounding 2^-b; a weight and the sum
of weights in fp32, each off by at most 2^-18 (|score| up to 4 in base 2, three
roundings of 2^-24 of it, the exponential's 2^-22, a sum of n terms); n terms
added in fp32, 2^-24 each; and of the output u |out|.  Bits b: a pair of bfloat16
numbers holds 16 (the upper cut, the lower rounded: 15 at worst), a pair of half
ones 22, one half 11."""
import numpy as np
import pytest
import torch

from tests.serving_ref import attention
from tests.test_gpu_tree_attention import causal, make, run

D, L = 64, 112
SCALE = 0.125


def pairs(T, hq, hkv, dtype, seed):
    """(q, kn, vn, k, v): scores in [-2, 2], pairs 1/128 or 2/128 apart."""
    rng = np.random.default_rng(seed)
    a = rng.integers(-240, 240, (L // 2, hkv)) / 16.0
    step = rng.choice([-2, -1, 1, 2], (L // 2, hkv)) / 16.0
    k = torch.zeros((L, hkv, D), dtype=torch.float64)
    k[0::2, :, 0], k[1::2, :, 0] = torch.from_numpy(a), torch.from_numpy(a + step)
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], (L // 2, hkv, D)))
    v = torch.stack([sign, -sign], 1).reshape(L, hkv, D)
    q = torch.zeros((T, hq, D), dtype=torch.float64)
    q[:, :, 0] = torch.from_numpy(rng.choice([-1.0, 0.75, 1.0], (T, hq)))
    kn, vn = torch.zeros((T, hkv, D)), torch.zeros((T, hkv, D))
    got = [x.to(dtype) for x in (q, kn, vn, k, v)]
    assert all(torch.equal(x.double(), y.double()) for x, y in zip((q, k, v), (got[0], got[3], got[4])))
    return got


def bound(ref, absum, dtype, bits, n):
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    return (2.0 ** -bits + 2 * 2.0 ** -18 + n * 2.0 ** -24) * absum + u * ref.abs() + (0 if dtype == torch.bfloat16 else 2.0 ** -25)


# rows a kv head: 5 and 16 (turned over), 24 and 150
CASES = [(5, 2, 2), (8, 4, 2), (6, 8, 2), (75, 4, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,hq,hkv", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_keep_their_bits(T, hq, hkv, dtype):
    q, kn, vn, k, v = pairs(T, hq, hkv, dtype, T)
    c = make([T], [L], hq, hkv, D, dtype, seed=T)
    ps = c["cache"].page_size
    for j in range(L // ps):
        page = int(c["cache"].page_table[0, j])
        for pool, x in ((c["cache"].k_pages, k), (c["cache"].v_pages, v)):
            pool[0, page] = x[j * ps:(j + 1) * ps].transpose(0, 1).cuda()
    c["q"] = q
    out, _ = run(c, kn=kn.cuda(), vn=vn.cuda(), scale=SCALE)
    ref, _, absum, _ = attention(q, kn, vn, k, v, causal([T])[0], SCALE)
    few = T * (hq // hkv) <= 16
    bits = 15 if dtype == torch.bfloat16 else 22 if few else 11
    err = (out.cpu().double() - ref).abs()
    tol = bound(ref, absum, dtype, bits, L + T)
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("T,hq,hkv", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_bound_tells_one_rounding_from_a_pair(T, hq, hkv, dtype):
    """Weights rounded once to the inputs' type, by the formula in 64 bits: far
    outside of the bound for a pair."""
    q, kn, vn, k, v = pairs(T, hq, hkv, dtype, T)
    ref, _, absum, _ = attention(q, kn, vn, k, v, causal([T])[0], SCALE)
    out = torch.zeros_like(ref)
    for t in range(T):
        for h in range(hq):
            g = h // (hq // hkv)
            a = torch.cat([k[:, g], kn[:t + 1, g]]).double() @ q[t, h].double() * SCALE
            w = torch.exp(a - a.max())
            out[t, h] = w.to(dtype).double() @ torch.cat([v[:, g], vn[:t + 1, g]]).double() / w.sum()
    over = (out - ref).abs() / bound(ref, absum, dtype, 15 if dtype == torch.bfloat16 else 22, L + T)
    assert float(over.max()) > 2
