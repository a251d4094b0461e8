"""Plain references, in 64 bits, of what a decoder does between the projections,
the attention and the verification.  No code of the package runs here."""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}  # half a step of subnormal numbers


def norm(v, kind, w, b, eps):
    """(normed v, how much of each value's terms an error of one part can move):
    for a relative error e of each operation the result is off by at most a few
    e times the second."""
    if kind == "none":
        return v, v.abs()
    off = v.abs().mean(-1, keepdim=True)
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    f = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    w = torch.ones_like(v[:1]) if w is None else w.double()
    b = torch.zeros_like(v[:1]) if b is None else b.double()
    y = v * f * w + b
    return y, y.abs() + b.abs() + w.abs() * f * (off if kind == "layer" else 0.0) + (v * f * w).abs()


def add_norm(x, residual, gate, post, pre, scale):
    """((r', its tolerance), (out, its tolerance)) in float64, but for the
    rounding to the outputs' types.  post, pre: (kind, w, b, eps).

    Every value is a chain of less than 2^7 operations of f32 (sums: up to 32
    elements a thread and ten steps of a tree; a reciprocal root of two units in
    the last place): each moves it by 2^-24 of the terms it is made of."""
    e = 2.0 ** -17
    v, terms = norm(x.double(), *post)
    if gate is not None:
        v, terms = v * gate.double(), terms * gate.double().abs()
    if residual is not None:
        v, terms = v + scale * residual.double(), terms + (scale * residual.double()).abs()
    kind, w, b, eps = pre
    out, more = norm(v, *pre)
    if kind == "none":
        return (v, e * terms), (out, e * terms)
    c = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    f = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    wa = 1.0 if w is None else w.double().abs()
    # an error of r' moves its own value, the mean, and the root mean square
    rms = torch.sqrt((terms * terms).mean(-1, keepdim=True))
    return (v, e * terms), (out, e * (more + wa * f * (terms + rms * (1 + (c * f).abs()))))


def close(got, want, tol, dtype=None):
    """got within tol plus its type's rounding of want; NaN and infinities alike."""
    dtype = got.dtype if dtype is None else dtype
    got, want, tol = got.double().cpu(), want.double().cpu(), torch.as_tensor(tol, dtype=torch.float64).cpu()
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN in other places"
    inf = ~finite & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), "infinities differ"
    bound = tol + HALF[dtype] * (want.abs() + tol) + TINY[dtype]
    bound = bound.expand_as(want) if bound.dim() else bound.repeat(want.shape)
    over = ((got - want).abs() - bound)[finite]
    assert not bool((over > 0).any()), f"{int((over > 0).sum())} of {over.numel()} too far off, by up to {float(over.max()):.3g}"


def rotary(x, positions, freq, rot, interleaved, scale=1.0, inverse=False):
    """(x turned, tolerance) in float64; x (n, heads, d).

    The angle enters the sine as a number of at most one half turn with 24 bits
    (2^-22.3 radians) and cosine and sine are off by two units in the last place:
    less than 2^-21 together.  Two products and their sum: 2^-22 more.  The
    reference's own angle is off by 2^-53 of itself."""
    x = x.double().cpu()
    a = positions.double().cpu()[:, None] * freq.double().cpu()
    off = (a.abs().amax(-1) if a.numel() else a.sum(-1)) * 2.0 ** -52 + 2.0 ** -20
    a = (-a if inverse else a)[:, None, :]
    u, v = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, s = a.cos() * scale, a.sin() * scale
    pair, size = [u * c - v * s, u * s + v * c], abs(scale) * (u.abs() + v.abs())
    join = (lambda p: torch.stack(p, -1).flatten(-2)) if interleaved else (lambda p: torch.cat(p, -1))
    y, tol = torch.cat([join(pair), x[..., rot:]], -1), torch.zeros_like(x)
    tol[..., :rot] = join([size, size]) * off[:, None, None]
    return y, tol


class Cache:
    """A paged cache as csgmv.h describes it, as lists of Python numbers: pages
    are given out lowest first, a shared page that is not full is copied before
    it is appended to."""

    def __init__(self, cache):
        self.ps, self.width = cache.page_size, cache.max_pages_per_seq
        self.table = cache.page_table.tolist()
        self.lens = cache.seq_lens.tolist()
        self.refs = cache.page_refs.tolist()

    def extend(self, seq, n):
        """[(slot)] of n more tokens, [(from page, to page, tokens)] of the copies."""
        old, copies = self.lens[seq], []
        need = math.ceil((old + n) / self.ps) - math.ceil(old / self.ps)
        free = [p for p, c in enumerate(self.refs) if c == 0]
        if n and old % self.ps:
            last = self.table[seq][old // self.ps]
            if self.refs[last] > 1:
                to = free.pop(0)
                self.refs[last] -= 1
                self.refs[to] = 1
                self.table[seq][old // self.ps] = to
                copies.append((last, to, old % self.ps))
        for i in range(need):
            page = free.pop(0)
            self.refs[page] = 1
            self.table[seq][math.ceil(old / self.ps) + i] = page
        self.lens[seq] = old + n
        return [self.table[seq][p // self.ps] * self.ps + p % self.ps for p in range(old, old + n)], copies


class Counts:
    """What a sequence's tokens are: times given, and which its prompt has."""

    def __init__(self):
        self.given, self.prompt = {}, set()

    def add(self, tokens, prompt=False):
        for v in tokens:
            if prompt:
                self.prompt.add(v)
            else:
                self.given[v] = self.given.get(v, 0) + 1

    def word(self, v):
        return self.given.get(v, 0) + (2 ** 30 if v in self.prompt else 0)

    def row(self, vocab):
        out = [0] * vocab
        for v in set(self.given) | self.prompt:
            out[v] = self.word(v)
        return out


def scores(logits, counts, branch, rho, alpha, beta, bias, allowed):
    """(z of one row in float64, how far rounding each step to f32 can move it).
    counts: Counts or None; branch: tokens; bias: [(token, value)]; allowed: bool
    (vocab,) or None."""
    z = logits.double().clone()
    size = torch.zeros_like(z)
    given, prompt = (dict(counts.given), counts.prompt) if counts else ({}, set())
    for v in branch:
        given[v] = given.get(v, 0) + 1
    for v in set(given) | set(prompt):
        x = float(z[v])
        x = x / rho if x > 0 else x * rho
        c = given.get(v, 0)
        s = 2 * abs(x) + (2 * abs(alpha) * c + abs(beta) + abs(x - alpha * c - beta) if c else 0.0)
        z[v], size[v] = x - (alpha * c + beta if c else 0.0), s
    for v, b in bias:
        z[v] += b
        size[v] += abs(float(z[v])) + abs(b)
    if allowed is not None:
        z[~allowed] = float("-inf")
    size[~torch.isfinite(z)] = 0.0
    return z, size.nan_to_num(0.0, 0.0, 0.0) * 2.0 ** -24


def distribution(z, off, temperature):
    """(probabilities, tolerance) of one row.  A relative error of a probability:
    of z and of the largest z over the temperature; of their difference and two
    factors (2^-22 of it); of the exponential and the division (2^-20); of the
    sum, weighted, of some 60 additions (2^-18)."""
    none = float("-inf")
    top = float(z.max())
    if bool(torch.isnan(z).any()) or (top == float("inf") and temperature > 0):
        return torch.full_like(z, float("nan")), 0.0
    if top == none:
        return torch.zeros_like(z), 0.0
    if temperature == 0:
        p = torch.zeros_like(z)
        p[int((z == top).nonzero()[0])] = 1.0
        return p, 0.0
    arg = (z - top) / temperature
    p = torch.softmax(z / temperature, -1)
    rel = (off + off.max()) / temperature + torch.where(torch.isfinite(arg), arg.abs(), 0.0) * 2.0 ** -22 + 2.0 ** -20
    return p, p * (rel + float((p * rel).sum()) + 2.0 ** -18) + 2.0 ** -140
