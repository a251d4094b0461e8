"""csgmv_add_norm against float64: types, widths from one element on, strides,
outputs in place of inputs, parts left out.  Tolerances: tests/step_ref.py."""
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.step_ref import add_norm, close

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def draw(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def side(g, kind, D, dtype, bias):
    """(Norm, what the reference takes of it)"""
    if kind == "none":
        return None, ("none", None, None, EPS)
    w = 1 + draw(g, (D,), dtype, 0.2)
    b = draw(g, (D,), dtype, 0.3) if bias else None
    return B.Norm(kind, w, b, eps=EPS), (kind, w, b, EPS)


def check(after, out, want, rtype):
    (r, rtol), (y, ytol) = want
    if after is not None:
        close(after, r, rtol, rtype)
    if out is not None:
        close(out, y, ytol)


@pytest.mark.parametrize("dtype,rtype", [(BF, BF), (BF, F32), (HF, HF), (HF, F32), (F32, F32)])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 63, 256, 264, 1001, 1024, 1032, 4096, 4097, 5120, 8192, 8200, 14336, 16383, 16384])
@pytest.mark.parametrize("n", [1, 5, 170])
def test_sums_and_norms(dtype, rtype, D, n):
    g = torch.Generator().manual_seed(D * 7 + n)
    pre_kind, post_kind = [("rms", "none"), ("layer", "rms"), ("rms", "layer"), ("layer", "layer")][(D + n) % 4]
    x, r = draw(g, (n, D), dtype), draw(g, (n, D), rtype, 3.0) + 0.5
    gate = None if (D + n) % 3 == 0 else draw(g, (n if (D + n) % 3 == 1 else 1, D), dtype)
    pre, pre_ref = side(g, pre_kind, D, dtype, n % 2)
    post, post_ref = side(g, post_kind, D, dtype, D % 2)
    after = torch.full_like(r, float("nan"))
    out = B.csgmv_add_norm(x, pre, residual=r, residual_out=after, post_norm=post, gate=gate, residual_scale=0.75)
    check(after, out, add_norm(x, r, gate, post_ref, pre_ref, 0.75), rtype)


@pytest.mark.parametrize("D", [64, 1000, 4096])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_rows_inside_wider_tensors(D, shift):
    """Strides that are no multiple of a vector, rows that begin anywhere;
    nothing around the rows is written."""
    g = torch.Generator().manual_seed(D + shift)
    n, dtype = 9, BF
    wide = [draw(g, (n + 1, D + 17 if shift == 1 else D + 24), dtype) for _ in range(5)]
    x, r, gate, after, out = (t[:n, shift:shift + D] for t in wide)
    before = [t.clone() for t in wide]
    pre, ref = side(g, "rms", D, dtype, False)
    B.csgmv_add_norm(x, pre, out, residual=r, residual_out=after, gate=gate)
    check(after, out, add_norm(before[0][:n, shift:shift + D], before[1][:n, shift:shift + D], before[2][:n, shift:shift + D],
                               ("none", None, None, EPS), ref, 1.0), dtype)
    for t, was in zip(wide, before):
        t[:n, shift:shift + D] = was[:n, shift:shift + D]
        assert torch.equal(t, was)


@pytest.mark.parametrize("dtype,D", [(BF, 4096), (F32, 520), (HF, 77)])
def test_in_place(dtype, D):
    g = torch.Generator().manual_seed(D)
    n = 33
    x, r = draw(g, (n, D), dtype), draw(g, (n, D), dtype)
    pre, ref = side(g, "layer", D, dtype, True)
    post, pref = side(g, "rms", D, dtype, False)
    want = add_norm(x.clone(), r.clone(), None, pref, ref, 0.5)
    got = B.csgmv_add_norm(x, pre, x, residual=r, post_norm=post, residual_scale=0.5)  # the residual too
    assert got is x
    check(r, x, want, dtype)
    # the sum over x, the norm over the residual
    x, r = draw(g, (n, D), dtype), draw(g, (n, D), dtype)
    want = add_norm(x.clone(), r.clone(), None, pref, ref, 1.0)
    B.csgmv_add_norm(x, pre, r, residual=r, residual_out=x, post_norm=post)
    check(x, r, want, dtype)


def test_parts_left_out():
    g = torch.Generator().manual_seed(0)
    n, D = 40, 520
    x, r = draw(g, (n, D), BF), draw(g, (n, D), F32)
    none = ("none", None, None, EPS)
    # a norm alone, without weights
    out = B.csgmv_add_norm(x, B.Norm("rms", eps=EPS))
    check(None, out, add_norm(x, None, None, none, ("rms", None, None, EPS), 1.0), BF)
    # the sum alone
    was = r.clone()
    assert B.csgmv_add_norm(x, None, residual=r, residual_scale=-2.0) is None
    check(r, None, add_norm(x, was, None, none, none, -2.0), F32)
    # a first residual
    first = torch.empty_like(r)
    out = B.csgmv_add_norm(x, B.Norm("layer", eps=EPS), residual_out=first)
    check(first, out, add_norm(x, None, None, none, ("layer", None, None, EPS), 1.0), F32)
    assert B.csgmv_add_norm(x[:0], B.Norm("rms")).shape == (0, D)


def test_a_norm_that_is_none_and_broadcast_rows():
    """kind "none" with an output: the sum, rounded; one row of x or of the residual
    for all (stride 0)."""
    g = torch.Generator().manual_seed(3)
    n, none = 50, ("none", None, None, EPS)
    for D in (4096, 1001):
        x, r = draw(g, (1, D), BF).expand(n, D), draw(g, (n, D), F32)
        after = torch.empty_like(r)
        out = B.csgmv_add_norm(x, B.Norm("none"), residual=r, residual_out=after, residual_scale=0.5)
        check(after, out, add_norm(x, r, None, none, none, 0.5), F32)
        pre, ref = side(g, "layer", D, BF, True)
        x, r = draw(g, (n, D), BF), draw(g, (1, D), BF).expand(n, D)
        after = torch.empty((n, D), dtype=BF, device="cuda")
        out = B.csgmv_add_norm(x, pre, residual=r, residual_out=after)
        check(after, out, add_norm(x, r, None, none, ref, 1.0), BF)


@pytest.mark.parametrize("rtype", [BF, F32])
@pytest.mark.parametrize("D", [513, 4097])
@pytest.mark.parametrize("shifts", [(0, 0, 0, 0), (3, 3, 3, 3), (1, 5, 5, 1), (1, 2, 3, 4)])
def test_rows_that_begin_anywhere(rtype, D, shifts):
    """Odd widths, each tensor's first row somewhere behind a boundary: alike, alike
    modulo the four elements of an f32 vector, or each elsewhere."""
    g = torch.Generator().manual_seed(D + sum(shifts))
    n, none = 21, ("none", None, None, EPS)

    def rows(shift, dtype):
        flat = draw(g, (n * D + 8,), dtype)
        return flat, flat[shift:shift + n * D].view(n, D)
    (fx, x), (fr, r), (fa, after), (fo, out) = rows(shifts[0], BF), rows(shifts[1], rtype), rows(shifts[2], rtype), rows(shifts[3], BF)
    was = fa.clone(), fo.clone()
    pre, ref = side(g, "rms", D, BF, True)
    B.csgmv_add_norm(x, pre, out, residual=r, residual_out=after)
    check(after, out, add_norm(x, r, None, none, ref, 1.0), rtype)
    for flat, old, k in ((fa, was[0], shifts[2]), (fo, was[1], shifts[3])):
        assert torch.equal(flat[:k], old[:k]) and torch.equal(flat[k + n * D:], old[k + n * D:])


def test_rows_of_one_value_and_of_infinities():
    """A centred norm of equal values is its bias; what is not finite stays in its row."""
    D = 1024
    x = torch.full((3, D), 7.0, dtype=F32, device="cuda")
    x[1, 5], x[2, 900] = float("inf"), float("nan")
    b = torch.arange(D, dtype=F32, device="cuda")
    out = B.csgmv_add_norm(x, B.Norm("layer", None, b, eps=EPS))
    assert torch.equal(out[0], b)
    assert bool(torch.isnan(out[1:]).all())


def test_large_and_small_values():
    """Mean squares far from one, in both directions, and a mean far above the deviation."""
    g = torch.Generator().manual_seed(5)
    none, D = ("none", None, None, EPS), 4096
    x = draw(g, (4, D), F32)
    x[0] *= 1e15
    x[1] *= 1e-12
    x[2] += 1000.0
    for kind in ("rms", "layer"):
        out = B.csgmv_add_norm(x, B.Norm(kind, eps=EPS))
        check(None, out, add_norm(x, None, None, none, (kind, None, None, EPS), 1.0), F32)


def test_a_captured_call_is_replayed():
    g = torch.Generator().manual_seed(1)
    x, r = draw(g, (64, 4096), BF), draw(g, (64, 4096), F32)
    pre, ref = side(g, "rms", 4096, BF, False)
    after, out = torch.empty_like(r), torch.empty_like(x)
    B.csgmv_add_norm(x, pre, out, residual=r, residual_out=after)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        B.csgmv_add_norm(x, pre, out, residual=r, residual_out=after)
    x.copy_(draw(g, (64, 4096), BF))
    r.copy_(draw(g, (64, 4096), F32))
    graph.replay()
    check(after, out, add_norm(x, r, None, ("none", None, None, EPS), ref, 1.0), F32)


def test_rows_past_32_bits_of_elements():
    """Offsets are 64 bits."""
    D, n = 16384, (1 << 31) // 16384 + 3
    x = torch.zeros((n, D), dtype=BF, device="cuda")
    x[-2:] = 1.0
    x[-1, ::2] = -3.0
    out = B.csgmv_add_norm(x, B.Norm("rms", eps=0.0), x)
    assert torch.equal(out[-2], torch.ones(D, dtype=BF, device="cuda"))
    want = torch.where(torch.arange(D, device="cuda") % 2 == 0, -3.0, 1.0).double() / 5 ** 0.5
    close(out[-1], want, 2.0 ** -17)


def laid_out(g, n, D, dtype, std=1.0, gap=0, shift=0):
    """Rows of D in a wider tensor of NaN that begin `shift` behind its boundary."""
    wide = torch.full((n * (D + gap) + 16,), float("nan"), dtype=dtype, device="cuda")
    rows = wide[shift:shift + n * (D + gap)].view(n, D + gap)[:, :D]
    rows.copy_(draw(g, (n, D), dtype, std))
    return wide, rows


# (rows, width, dtype, residual, post, pre, gate, gap, shift): several rows to a CTA, its
# inputs asked for while the one before is worked on, and the same rows one by one
MANY = [
    (2500, 4096, BF, BF, "none", "rms", None, 0, 0),
    (2501, 4104, HF, HF, "layer", "none", None, 8, 0),
    (700, 8200, BF, F32, "rms", "layer", None, 0, 0),
    (615, 16384, HF, HF, "rms", "rms", "column", 0, 0),
    (1300, 10008, BF, None, "none", "layer", None, 8, 8),
    (1300, 6144, BF, BF, "none", "rms", None, 0, 0),
    (5000, 513, BF, F32, "layer", "layer", "token", 0, 0),
    (2500, 1001, HF, HF, "none", "rms", "column", 0, 3),
    (900, 4097, BF, BF, "rms", "layer", "token", 0, 0),
    (900, 4096, BF, BF, "none", "rms", "token", 5, 1),
    (470, 16371, BF, F32, "none", "rms", "token", 0, 5),
    (900, 4097, F32, F32, "rms", "rms", "token", 0, 0),
    (40001, 40, BF, BF, "none", "layer", "column", 0, 0),
    (9001, 129, HF, F32, "rms", "rms", "token", 0, 0),
    (9001, 128, BF, BF, "none", "rms", None, 0, 0),
    (3001, 7, F32, F32, "none", "layer", "token", 0, 0),
]


@pytest.mark.parametrize("n,D,dtype,rtype,post,pre,gate,gap,shift", MANY)
def test_many_rows(n, D, dtype, rtype, post, pre, gate, gap, shift):
    """What lies before, between and behind the rows is NaN, and stays; some rows hold
    one, which stays in its row."""
    g = torch.Generator().manual_seed(n + D)
    xw, x = laid_out(g, n, D, dtype, gap=gap, shift=shift)
    x[5::97, D - 1], x[6::97, 0] = float("nan"), float("inf")
    rw, r = laid_out(g, n, D, rtype, 3.0, gap=gap, shift=shift) if rtype else (None, None)
    gw, gt = (None, None) if gate is None else laid_out(g, 1 if gate == "column" else n, D, dtype, gap=gap, shift=shift)
    pre, pre_ref = side(g, pre, D, dtype, D % 3 == 0)
    post, post_ref = side(g, post, D, dtype, D % 2 == 1)
    ow, out = laid_out(g, n, D, dtype, gap=gap, shift=shift)
    aw, after = laid_out(g, n, D, rtype or dtype, gap=gap, shift=shift)
    B.csgmv_add_norm(x, pre, out, residual=r, residual_out=after, post_norm=post, gate=gt, residual_scale=0.75)
    want = add_norm(x, r, gt, post_ref, pre_ref, 0.75)
    check(after, out, want, rtype or dtype)
    once = out.clone(), after.clone()
    for wide, rows in ((ow, out), (aw, after)):
        rows.fill_(float("nan"))
        assert bool(torch.isnan(wide).all())
    # single rows, and rows in place of the inputs
    for k in (0, 1, n // 2, n - 1):
        one = slice(k, k + 1)
        B.csgmv_add_norm(x[one], pre, out[one], residual=None if r is None else r[one], residual_out=after[one], post_norm=post,
                         gate=gt if gate != "token" else gt[one], residual_scale=0.75)
        check(after[one], out[one], [(v[one], t[one]) for v, t in want], rtype or dtype)
    if r is not None:
        B.csgmv_add_norm(x, pre, x, residual=r, post_norm=post, gate=gt, residual_scale=0.75)
        assert torch.equal(x.nan_to_num(), once[0].nan_to_num()) and torch.equal(r.nan_to_num(), once[1].nan_to_num())


@pytest.mark.parametrize("D", [4096, 4097])
def test_one_row_of_an_input_for_many(D):
    """A stride of 0, where several rows come to a CTA one behind the other."""
    g = torch.Generator().manual_seed(D)
    n, none = 2600, ("none", None, None, EPS)
    pre, ref = side(g, "rms", D, BF, False)
    one, many = draw(g, (D + 3,), BF), draw(g, (n, D), BF)
    for off in (0, 3) if D % 8 else (0,):
        row = one[off:off + D].view(1, D).expand(n, D)
        for x, r in ((row, many), (many, row)):
            after = torch.empty((n, D), dtype=BF, device="cuda")
            out = B.csgmv_add_norm(x, pre, residual=r, residual_out=after)
            check(after, out, add_norm(x, r, None, none, ref, 1.0), BF)
