"""Attention of draft trees over the paged cache against a plain float64
reference.

Tolerance, from the arithmetic: with u = 2^-9 (bf16) or 2^-11 (f16) the weights
and the output are each rounded once (u |w||v| summed, u |out|); a score of D
products summed in fp32 is off by at most (D + 16) 2^-24 sum |q||k| scale, which
moves a weight and the sum of weights by that much relatively, and the
exponentials and sums in fp32 by less than 2^-18; f16 weights below its normal
range are rounded in steps of at most 2^-28 of the largest weight."""
import numpy as np
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_i32
from tests.serving_ref import attention, pack_bits, tree_bits

pytestmark = pytest.mark.gpu


def make(T, L, hq, hkv, d, dtype=torch.bfloat16, ps=16, layout="HND", seed=0, qstd=1.0, extra_pages=3, poison=True,
         slots=None, kstd=1.0):
    """Requests with T[b] rows over L[b] cached tokens; pages scattered, page
    slots past a sequence's end NaN."""
    g = torch.Generator()
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = [-(-n // ps) for n in L]
    pages = sum(need) + extra_pages
    seqs = len(L) if slots is None else max(slots) + 1
    order = rng.permutation(pages)
    table = np.full((seqs, max(1, max(need))), -1, np.int32)
    lens = np.zeros(seqs, np.int32)
    shape = (1, pages, hkv, ps, d) if layout == "HND" else (1, pages, ps, hkv, d)
    kp = torch.full(shape, float("nan") if poison else 0.0, dtype=dtype)
    vp = kp.clone()
    ctx, at = [], 0
    for b, n in enumerate(L):
        k = (torch.randn((n, hkv, d), generator=g) * kstd).to(dtype)
        v = torch.randn((n, hkv, d), generator=g).to(dtype)
        s = b if slots is None else slots[b]
        lens[s] = n
        for j in range(need[b]):
            p = int(order[at])
            at += 1
            table[s, j] = p
            m = min(ps, n - j * ps)
            for pool, x in ((kp, k), (vp, v)):
                if layout == "HND":
                    pool[0, p, :, :m] = x[j * ps:j * ps + m].transpose(0, 1)
                else:
                    pool[0, p, :m] = x[j * ps:j * ps + m]
        ctx.append((k, v))
    N = sum(T)
    q = (torch.randn((N, hq, d), generator=g) * qstd).to(dtype)
    kn = (torch.randn((N, hkv, d), generator=g) * kstd).to(dtype)
    vn = torch.randn((N, hkv, d), generator=g).to(dtype)
    cache = B.KvCache(kp.cuda(), vp.cuda(), dev_i32(table), dev_i32(lens),
                      torch.ones(pages, dtype=torch.int32, device="cuda"), layout=layout)
    indptr = np.concatenate([[0], np.cumsum(T)]).astype(np.int32)
    return dict(cache=cache, q=q, kn=kn, vn=vn, ctx=ctx, T=T, L=L, indptr=indptr, slots=slots, d=d, dtype=dtype)


def run(c, mask=None, q=None, kn=None, vn=None, scale=None, stream=None):
    q = c["q"].cuda() if q is None else q
    out = torch.full(tuple(q.shape), 7.0, dtype=c["dtype"], device="cuda")
    lse = torch.full(tuple(q.shape[:2]), 7.0, dtype=torch.float32, device="cuda")
    B.csgmv_tree_attention(q, c["kn"].cuda() if kn is None else kn, c["vn"].cuda() if vn is None else vn, c["cache"], 0,
                           dev_i32(c["indptr"]), out, mask=None if mask is None else dev_i32(mask),
                           seq_slots=None if c["slots"] is None else dev_i32(c["slots"]), scale=scale, lse=lse)
    torch.cuda.synchronize()
    return out, lse


def compare(c, got, sees, scale=None):
    out, lse = (t.cpu() for t in got)
    scale = c["d"] ** -0.5 if scale is None else scale
    u = 2.0 ** -9 if c["dtype"] == torch.bfloat16 else 2.0 ** -11
    for b, (k, v) in enumerate(c["ctx"]):
        lo, hi = c["indptr"][b], c["indptr"][b + 1]
        if lo == hi:
            continue
        ref, rl, absum, big = attention(c["q"][lo:hi], c["kn"][lo:hi], c["vn"][lo:hi], k, v, sees[b], scale)
        off = (c["d"] + 16) * 2.0 ** -24 * big + 2.0 ** -18
        n = k.shape[0] + hi - lo
        tol = u * absum * 1.01 + u * ref.abs() * 1.01 + 2 * off * absum + (0 if u > 2 ** -10 else 2.0 ** -24 + n * 2.0 ** -26)
        err = (out[lo:hi].double() - ref).abs()
        assert (err <= tol).all(), (b, float((err - tol).max()), float(err.max()))
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse[lo:hi]), empty) and (lse[lo:hi][empty] < 0).all()
        le = (lse[lo:hi].double() - rl)[~empty].abs()
        assert (le <= off + 2.0 ** -22 * rl[~empty].abs()).all(), (b, float(le.max()))
        assert (out[lo:hi][empty] == 0).all()


def causal(T):
    return [torch.ones((t, t), dtype=torch.bool).tril() for t in T]


def random_parents(rng, n):
    return [-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, n)]


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,ps", [(64, 8), (64, 64), (128, 16), (128, 32), (128, 128), (64, 256)])
def test_decode_lengths(d, ps, dtype, layout):
    """One token a request over every length around a page and a tile."""
    L = [0, 1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 120, 121, 127, 128, 129, 255, 256, 257, 500, 1023]
    c = make([1] * len(L), L, 4, 2, d, dtype, ps, layout, seed=d + ps)
    got = run(c)
    assert c["cache"].device_status() == 0
    compare(c, got, causal(c["T"]))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (3, 1), (8, 1), (20, 4), (128, 1), (6, 2)])
def test_head_groups(hq, hkv):
    c = make([1, 5, 2, 0, 9], [33, 0, 130, 40, 257], hq, hkv, 64, seed=hq)
    compare(c, run(c), causal(c["T"]))


@pytest.mark.parametrize("T", [[1, 16, 17, 31, 32, 33, 64], [127, 128, 129], [300], [2, 0, 0, 1]])
@pytest.mark.parametrize("d", [64, 128])
def test_causal_rows(T, d):
    """Many rows with no mask: prompts, with and without a cached prefix."""
    L = [(37 * i) % 200 for i in range(len(T))]
    c = make(T, L, 4, 2, d, seed=sum(T))
    compare(c, run(c), causal(T))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,words", [([1, 5, 12, 32], 1), ([33, 64, 40], 2), ([70, 96, 3], 3), ([200, 256], 8)])
def test_trees(sizes, words, dtype):
    """Trees at every offset of the cached length against a tile; bits past a
    request's rows are ignored."""
    rng = np.random.default_rng(words)
    L = [5, 121, 130, 64][:len(sizes)]
    c = make(sizes, L, 8, 2, 128, dtype, seed=words, qstd=2.0)
    sees = [tree_bits(random_parents(rng, n)) for n in sizes]
    mask = np.concatenate([pack_bits(s, words, junk=0x5a5a5a5a5a5a) for s in sees])
    compare(c, run(c, mask), sees)


def test_rows_that_see_nothing():
    """A mask without a bit, over no cached tokens: zeros and -inf; over cached
    tokens: those alone."""
    rng = np.random.default_rng(0)
    sizes, L = [6, 40, 3], [0, 0, 19]
    c = make(sizes, L, 4, 1, 64, seed=4)
    sees = [torch.from_numpy(rng.random((n, n)) < 0.3) for n in sizes]
    for s in sees:
        s[::2] = False
    got = run(c, np.concatenate([pack_bits(s, 2) for s in sees]))
    compare(c, got, sees)
    assert torch.isinf(got[1][0]).all() and (got[0][0] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_masked_rows_hold_anything(value, dtype):
    """Drafted rows that hold NaN or infinity reach those that see them only."""
    rng = np.random.default_rng(1)
    sizes, L = [20, 9], [130, 0]
    c = make(sizes, L, 8, 2, 64, dtype, seed=8)
    sees = [tree_bits(random_parents(rng, n)) for n in sizes]
    mask = np.concatenate([pack_bits(s, 1) for s in sees])
    clean = run(c, mask)
    kn, vn = c["kn"].clone(), c["vn"].clone()
    kn[4, 0, 3] = value
    vn[7, 1, :5] = value
    vn[25, 0, 60] = value
    out, lse = run(c, mask, kn=kn.cuda(), vn=vn.cuda())
    reach = torch.zeros((29, 8), dtype=torch.bool)
    for b, rows, head in ((0, 4, slice(0, 4)), (0, 7, slice(4, 8)), (1, 5, slice(0, 4))):
        base = c["indptr"][b]
        reach[base:base + sizes[b], head] |= sees[b][:, rows][:, None]
    keep = (~reach).cuda()
    assert torch.equal(out[keep], clean[0][keep])
    # a row that does see them shows it: value v at 7 and 25
    for row, head, el in ((7, 4, 0), (25, 0, 60)):
        x = float(out[row, head, el])
        assert x == value or (np.isnan(value) and np.isnan(x))
    if not np.isnan(value):
        assert torch.equal(lse[7], clean[1][7])


def test_the_types_lowest_value_and_infinite_scores():
    """A cached key that scores -inf or the lowest finite number counts for
    nothing beside others; alone with -inf it gives an empty row's answer."""
    c = make([1, 1], [3, 1], 1, 1, 64, seed=2, poison=False)
    q = torch.ones((2, 1, 64), dtype=torch.bfloat16)
    kn = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    kn[1] = float("-inf")
    c["q"], c["kn"] = q, kn
    pool = c["cache"].k_pages
    table = c["cache"].page_table.cpu()
    pool[0, int(table[0, 0]), 0, 0] = torch.finfo(torch.bfloat16).min
    pool[0, int(table[0, 0]), 0, 1] = float("-inf")
    pool[0, int(table[1, 0]), 0, 0] = float("-inf")
    out, lse = run(c, mask=np.array([[1], [1]], np.int32))
    k2 = pool[0, int(table[0, 0]), 0, 2].cpu().double()
    a = torch.stack([k2.sum() / 8, torch.zeros((), dtype=torch.float64)])
    w = torch.softmax(a, 0)
    want = w[0] * c["ctx"][0][1][2, 0].double() + w[1] * c["vn"][0, 0].double()
    assert torch.allclose(out[0, 0].cpu().double(), want, rtol=2 ** -7, atol=2 ** -7)
    assert float(lse[1, 0]) == float("-inf") and (out[1] == 0).all()


def test_strides_slots_streams_and_scale():
    """q, k, v as slices of one projection, sequences in other slots, another
    stream, another scale."""
    slots = [5, 0, 3]
    c = make([4, 7, 1], [50, 0, 200], 8, 2, 128, seed=11, slots=slots)
    wide = torch.cat([c["q"].reshape(12, -1), c["kn"].reshape(12, -1), c["vn"].reshape(12, -1)], 1).cuda()
    q = wide[:, :1024].view(12, 8, 128)
    kn, vn = wide[:, 1024:1280].view(12, 2, 128), wide[:, 1280:].view(12, 2, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(c, q=q, kn=kn, vn=vn, scale=0.3)
    compare(c, got, causal(c["T"]), scale=0.3)


def test_padded_pools_and_outputs():
    """Pools with room between heads, an output inside a wider buffer."""
    c = make([3, 1], [70, 16], 4, 2, 64, seed=12)
    for name in ("k_pages", "v_pages"):
        src = getattr(c["cache"], name)
        big = torch.full((1, src.shape[1] + 1, 3, 16, 72), float("nan"), dtype=src.dtype, device="cuda")
        view = big[:, :src.shape[1], :2, :, :64]
        view.copy_(src)
        c[name] = view
    old = c["cache"]
    c["cache"] = B.KvCache(c["k_pages"], c["v_pages"], old.page_table, old.seq_lens, old.page_refs)
    buf = torch.full((4, 6, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 1:5]
    lse = torch.empty((4, 4), dtype=torch.float32, device="cuda")
    B.csgmv_tree_attention(c["q"].cuda(), c["kn"].cuda(), c["vn"].cuda(), c["cache"], 0, dev_i32(c["indptr"]), out, lse=lse)
    torch.cuda.synchronize()
    compare(c, (out, lse), causal(c["T"]))
    assert (buf[:, 0] == 3).all() and (buf[:, 5] == 3).all()


@pytest.mark.parametrize("T,L,hkv", [([1], [40000], 1), ([9, 3], [20011, 5], 2), ([64], [9000], 1)])
def test_long_axis_split_over_the_gpu(T, L, hkv):
    """Few rows over many tokens, so the axis is cut and joined again; scores
    that grow along it."""
    c = make(T, L, 4 * hkv, hkv, 128, seed=L[0], qstd=3.0, ps=64)
    got = run(c)
    compare(c, got, causal(T))
    again = run(c)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,L", [
    ([64, 64, 70, 2, 33], [3000, 2500, 300, 50, 4000]),  # one to three row tiles, the second of 4 rows
    ([0, 63, 1, 36, 36, 0], [9, 1024, 5000, 129, 0, 64]),  # the second of 16, a request before and after without rows
    ([128], [20000]), ([64] * 40, [100 + 37 * i for i in range(40)])])
def test_heads_of_several_row_tiles(T, L, d, dtype):
    """Row tiles of a head that CTAs take together, and ones that are missing
    there or small."""
    c = make(T, L, 8, 2, d, dtype, ps=32, layout="NHD", seed=len(T) + d, qstd=1.5)
    compare(c, run(c), causal(T))


@pytest.mark.parametrize("T,hq", [([1], 4), ([9], 8), ([1, 9, 33], 8)])
def test_many_items_of_several_tiles(T, hq):
    """Ten and more items a CTA, most of two to five token tiles."""
    n = 800
    T = [T[i % len(T)] for i in range(n)]
    c = make(T, [130 + (97 * i) % 500 for i in range(n)], hq, 2, 64, seed=hq)
    compare(c, run(c), causal(T))
    assert c["cache"].device_status() == 0


def test_growing_and_falling_scores():
    """Rows whose maximum moves by hundreds along the tokens, both ways."""
    c = make([2, 2], [700, 700], 2, 1, 64, torch.float16, seed=21, poison=False)
    ramp = torch.linspace(-40, 40, 700)
    for b, sign in ((0, 1.0), (1, -1.0)):
        k = torch.zeros((700, 1, 64))
        k[:, 0, 0] = sign * ramp
        c["ctx"][b] = (k.half(), c["ctx"][b][1])
        for i in range(700):
            c["cache"].k_pages[0, int(c["cache"].page_table[b, i // 16]), 0, i % 16] = k[i, 0].half().cuda()
    c["q"].zero_()
    c["q"][:, :, 0] = 16.0
    compare(c, run(c), causal(c["T"]))


def test_many_requests_and_empty_batches():
    rng = np.random.default_rng(7)
    T = [int(x) for x in rng.integers(0, 3, 700)]
    L = [int(x) for x in rng.integers(0, 40, 700)]
    c = make(T, L, 2, 1, 64, seed=7)
    compare(c, run(c), causal(T))
    e = make([0, 0], [5, 0], 2, 1, 64)
    run(e)
    assert e["cache"].device_status() == 0


def test_pool_beyond_32_bit_offsets():
    pages = (1 << 31) // (16 * 8 * 128) + 64
    cache = B.KvCache.allocate(1, pages, 16, 8, 128, 1, 4)
    k, v = (torch.randn((50, 8, 128), generator=torch.Generator().manual_seed(s)).bfloat16() for s in (1, 2))
    table = [pages - 1, 3, pages - 7, pages - 2]
    for j, p in enumerate(table):
        m = min(16, 50 - 16 * j)
        cache.k_pages[0, p, :, :m] = k[16 * j:16 * j + m].transpose(0, 1).cuda()
        cache.v_pages[0, p, :, :m] = v[16 * j:16 * j + m].transpose(0, 1).cuda()
    cache.page_table.copy_(dev_i32([table]))
    cache.seq_lens.fill_(50)
    c = dict(cache=cache, q=torch.randn((2, 8, 128)).bfloat16(), kn=torch.randn((2, 8, 128)).bfloat16(),
             vn=torch.randn((2, 8, 128)).bfloat16(), ctx=[(k, v)], T=[2], L=[50], indptr=np.array([0, 2], np.int32),
             slots=None, d=128, dtype=torch.bfloat16)
    compare(c, run(c), causal([2]))


def test_bad_requests_are_left_out():
    """A slot out of range, a negative length, more rows than mask bits: their
    rows keep what they held, the others are right."""
    c = make([2, 2, 33, 2], [20, 20, 20, 20], 2, 1, 64, seed=3, slots=[0, 1, 2, 3])
    c["cache"].seq_lens[1] = -4
    c["slots"] = [9, 1, 2, 3]
    sees = causal(c["T"])
    mask = np.concatenate([np.zeros((n, 1), np.int32) if n > 32 else pack_bits(s, 1) for s, n in zip(sees, c["T"])])
    out, lse = run(c, mask)
    assert c["cache"].device_status() & 1 and c["cache"].device_status() & 8
    assert (out[:37] == 7).all() and (lse[:37] == 7).all()
    ref, _, _, _ = attention(c["q"][37:], c["kn"][37:], c["vn"][37:], *c["ctx"][3], sees[3], 64 ** -0.5)
    assert (out[37].cpu().double() - ref[0]).abs().max() < 0.05


def test_refusals():
    c = make([1], [4], 2, 1, 64)
    q, kn, vn, ptr = c["q"].cuda(), c["kn"].cuda(), c["vn"].cuda(), dev_i32([0, 1])
    out = torch.empty_like(q)

    def call(**kw):
        a = dict(q=q, kn=kn, vn=vn, layer=0, out=out)
        a.update(kw)
        opt = {k: v for k, v in a.items() if k not in ("q", "kn", "vn", "layer", "out")}
        B.csgmv_tree_attention(a["q"], a["kn"], a["vn"], c["cache"], a["layer"], ptr, a["out"], **opt)

    for kw, msg in ((dict(q=q.half()), "type"), (dict(layer=1), "layer"), (dict(scale=0.0), "scale"),
                    (dict(scale=float("nan")), "scale"), (dict(kn=kn.float(), vn=vn.float()), "type"),
                    (dict(mask=torch.zeros((2, 1), dtype=torch.int32, device="cuda")), "mask"),
                    (dict(lse=torch.zeros((1, 1), device="cuda")), "lse"), (dict(out=out[:, :1]), "tokens, heads")):
        with pytest.raises(B.CsgmvError, match=msg):
            call(**kw)
    with pytest.raises(B.CsgmvError, match="multiple of num_kv_heads"):
        e = make([1], [4], 3, 2, 64)
        run(e)
    with pytest.raises(B.CsgmvError, match="head_dim"):
        run(make([1], [4], 2, 1, 32))
    assert c["cache"].device_status() == 0
