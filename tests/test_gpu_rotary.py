"""csgmv_rotary against float64: types, layouts, parts of a head, far positions,
strides, outputs in place.  Tolerances: tests/step_ref.py."""
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.step_ref import close, rotary

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SCALINGS = [None, ("linear", 4.0), ("ntk", 2.0), ("wavelength", 8.0, 1.0, 4.0, 8192.0), ("yarn", 4.0, 8192.0)]


def draw(g, shape, dtype):
    return torch.randn(shape, generator=g).to(dtype).cuda()


def positions(g, n, most):
    return torch.randint(0, most, (n,), generator=g, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(2, 2), (5, 4), (64, 64), (80, 20), (80, 80), (96, 48), (128, 128), (128, 32), (100, 100), (192, 64),
                                   (256, 256), (1024, 1024), (1023, 1022), (64, 0)])
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (3, 5, 0), (37, 8, 2), (513, 20, 4)])
def test_heads(dtype, interleaved, d, rot, n, hq, hk):
    g = torch.Generator().manual_seed(d * 1000 + rot + n)
    rope = B.Rope(d, rotary_dim=rot, interleaved=interleaved, scaling=SCALINGS[(n + d) % 5] if rot > 2 else None)
    q, k = draw(g, (n, hq, d), dtype), draw(g, (n, hk, d), dtype) if hk else None
    pos = positions(g, n, 100000)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan")) if hk else None
    inverse = n % 2 == 0
    B.csgmv_rotary(rope, pos, q, k, q_out=qo, k_out=ko, inverse=inverse)
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            close(y, *rotary(x, pos, rope.freq, rot, interleaved, rope.scale, inverse))
            assert torch.equal(y[..., rot:], x[..., rot:])
    # in place gives the same bits
    if hk:
        B.csgmv_rotary(rope, pos, q, k, inverse=inverse)
        assert torch.equal(q, qo) and torch.equal(k, ko)
    else:
        B.csgmv_rotary(rope, pos, q, inverse=inverse)
        assert torch.equal(q, qo)


@pytest.mark.parametrize("n", [7, 20011])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_one_projection(n, off, dtype):
    """q and k side by side in rows that begin anywhere, turned in place: the
    values beside them, and around, stay."""
    g = torch.Generator().manual_seed(n + off)
    hq, hk, d = 8, 2, 64
    wide = torch.randn((n, (hq + 2 * hk) * d + 3 * off), generator=g).to(dtype).cuda()
    was = wide.clone()
    body = wide[:, off:off + (hq + 2 * hk) * d]
    q, k = body[:, :hq * d].view(n, hq, d) if off == 0 else body[:, :hq * d].unflatten(1, (hq, d)), \
        body[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    pos = positions(g, n, 4096)
    rope = B.Rope(d)
    B.csgmv_rotary(rope, pos, q, k)
    old = was[:, off:off + (hq + 2 * hk) * d]
    close(q, *rotary(old[:, :hq * d].unflatten(1, (hq, d)), pos, rope.freq, d, False))
    close(k, *rotary(old[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)), pos, rope.freq, d, False))
    wide[:, off:off + (hq + hk) * d] = was[:, off:off + (hq + hk) * d]
    assert torch.equal(wide, was)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 32), (80, 20), (72, 64), (70, 32), (64, 0)])
def test_parts_of_heads_in_place_and_apart(dtype, interleaved, d, rot):
    """Queries in place with keys apart, keys in place with queries apart, or
    queries alone: what is not turned keeps its bits, whatever they are."""
    g = torch.Generator().manual_seed(d + rot)
    n, rope = 130, B.Rope(d, rotary_dim=rot, interleaved=interleaved)
    pos = positions(g, n, 30000)
    bits = torch.int16 if dtype is BF else torch.int32
    for q_apart, k_apart in ((False, True), (True, False), (False, None), (False, False)):
        q, k = draw(g, (n, 6, d), dtype), draw(g, (n, 3, d), dtype)
        for x in (q, k):
            x.view(bits)[..., rot:] = torch.randint(-2 ** 15, 2 ** 15, (n, x.shape[1], d - rot), generator=g, dtype=bits).cuda()
        was = q.clone(), k.clone()
        qo, ko = torch.empty_like(q) if q_apart else q, torch.empty_like(k) if k_apart else k
        B.csgmv_rotary(rope, pos, q, None if k_apart is None else k, q_out=qo, k_out=None if k_apart is None else ko)
        for x, y, turned in ((was[0], qo, True), (was[1], ko, k_apart is not None)):
            if turned:
                close(y[..., :rot], *(t[..., :rot] for t in rotary(x.nan_to_num(), pos, rope.freq, rot, interleaved)))
                assert torch.equal(y.view(bits)[..., rot:], x.view(bits)[..., rot:])
            else:
                assert torch.equal(y.view(bits), x.view(bits))
        for x, y, apart in ((was[0], q, q_apart), (was[1], k, k_apart)):
            if apart:
                assert torch.equal(x.view(bits), y.view(bits))


def test_heads_outside_the_tokens():
    """(heads, tokens, d) seen as (tokens, heads, d); a head broadcast over many."""
    g = torch.Generator().manual_seed(2)
    q = draw(g, (6, 50, 64), BF).transpose(0, 1)
    one = draw(g, (50, 1, 64), BF)
    k = one.expand(50, 3, 64)
    pos, rope = positions(g, 50, 9000), B.Rope(64, interleaved=True)
    qo, ko = torch.empty((6, 50, 64), dtype=BF, device="cuda").transpose(0, 1), torch.empty((50, 3, 64), dtype=BF, device="cuda")
    B.csgmv_rotary(rope, pos, q, k, q_out=qo, k_out=ko)
    close(qo, *rotary(q, pos, rope.freq, 64, True))
    close(ko, *rotary(k, pos, rope.freq, 64, True))


def test_far_and_negative_positions():
    """No angle loses bits: neighbouring positions near 2^31 differ by one step, and
    position 0 leaves all as it is."""
    g = torch.Generator().manual_seed(4)
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, -2 ** 24, 2 ** 30, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    n, d = pos.numel(), 128
    q = draw(g, (n, 4, d), F32)
    rope = B.Rope(d, base=500000.0)
    out = torch.empty_like(q)
    B.csgmv_rotary(rope, pos, q, q_out=out)
    close(out, *rotary(q, pos, rope.freq, d, False))
    assert torch.equal(out[0], q[0])
    # the relative turn of neighbours is that of one position, wherever they are
    far = torch.tensor([2 ** 31 - 2, 2 ** 31 - 1], dtype=torch.int32).cuda()
    same = q[:1].expand(2, 4, d).contiguous()
    a = torch.empty_like(same)
    B.csgmv_rotary(rope, far, same, q_out=a)
    B.csgmv_rotary(rope, torch.ones(1, dtype=torch.int32, device="cuda"), a[:1])
    tol = 2.0 ** -19 * (a[:1, :, :64].abs() + a[:1, :, 64:].abs() + a[1:, :, :64].abs() + a[1:, :, 64:].abs()).repeat(1, 1, 2)
    close(a[:1], a[1:], tol)


def test_small_angles_keep_their_bits():
    """Of a pair (0, 1) a small angle's sine is left: an angle in f32 and a sine of two
    units in the last place, 2^-21 of it, however small (2^-64 turns: a radian is
    2^61.3 of them)."""
    f = torch.tensor([2.0 ** -k for k in range(2, 34)], dtype=torch.float64)
    rope = B.Rope(64, freq=f)
    x = torch.zeros((3, 1, 64), dtype=F32, device="cuda")
    x[..., 32:] = 1.0
    pos = torch.tensor([1, -1, 3], dtype=torch.int32, device="cuda")
    B.csgmv_rotary(rope, pos, x)
    want = -torch.sin(pos.double().cpu()[:, None] * f)
    close(x[:, 0, :32], want, 2.0 ** -21 * want.abs() + 2.0 ** -61)


def test_the_inverse_is_the_gradient():
    """<g, R x> = <R^T g, x>, and turning there and back is scale^2."""
    g = torch.Generator().manual_seed(6)
    n, d = 64, 96
    rope = B.Rope(d, rotary_dim=48, scaling=("yarn", 8.0, 4096))
    pos = positions(g, n, 40000)
    x, go = draw(g, (n, 3, d), F32), draw(g, (n, 3, d), F32)
    y, gx = torch.empty_like(x), torch.empty_like(x)
    B.csgmv_rotary(rope, pos, x, q_out=y)
    B.csgmv_rotary(rope, pos, go, q_out=gx, inverse=True)
    a, b = (go.double() * y.double()).sum((1, 2)), (gx.double() * x.double()).sum((1, 2))
    size = (go.double().abs() * rope.scale * 2).sum((1, 2)) * x.double().abs().amax((1, 2))
    assert bool(((a - b).abs() <= 2.0 ** -19 * size).all())
    # differences of the forward pass: it is linear, so they are exact up to rounding
    B.csgmv_rotary(rope, pos, y, inverse=True)
    want = x.double().clone()
    want[..., :48] *= rope.scale ** 2
    close(y, want, 2.0 ** -18 * rope.scale ** 2 * 2 * x.double().abs().amax(-1, keepdim=True))


def test_rounding_is_once():
    """Where the turned value is known to float32, bf16 and half results are it, rounded."""
    g = torch.Generator().manual_seed(8)
    pos, rope = positions(g, 200, 131072), B.Rope(128)
    for dtype in (BF, HF):
        q = draw(g, (200, 4, 128), dtype)
        full, low = q.float(), q.clone()
        B.csgmv_rotary(rope, pos, full)
        B.csgmv_rotary(rope, pos, low)
        assert torch.equal(low, full.to(dtype))


def test_a_captured_call_is_replayed():
    g = torch.Generator().manual_seed(9)
    rope, pos = B.Rope(128), positions(g, 100, 8192)
    q, k = draw(g, (100, 8, 128), BF), draw(g, (100, 2, 128), BF)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    B.csgmv_rotary(rope, pos, q, k, q_out=qo, k_out=ko)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        B.csgmv_rotary(rope, pos, q, k, q_out=qo, k_out=ko)
    q.copy_(draw(g, (100, 8, 128), BF))
    pos.copy_(positions(g, 100, 8192))
    graph.replay()
    close(qo, *rotary(q, pos, rope.freq, 128, False))
    close(ko, *rotary(k, pos, rope.freq, 128, False))


def test_offsets_past_32_bits():
    n, hq, d = 70000, 40, 1024  # 2.9e9 elements
    q = torch.zeros((n, hq, d), dtype=BF, device="cuda")
    q[-1, -1] = 1.0
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos[-1] = 3
    rope = B.Rope(d)
    B.csgmv_rotary(rope, pos, q)
    close(q[-1:, -1:], *rotary(torch.ones((1, 1, d)), pos[-1:], rope.freq, d, False))
    assert not bool(q[:-1].any()) and not bool(q[-1, :-1].any())
