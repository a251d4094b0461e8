"""Plain references of the serving step's operators: attention and the
verification walk in 64 bits, the paged cache as lists of tokens.  No code of
the package runs here."""
from __future__ import annotations

import numpy as np
import torch


def attention(q, k_new, v_new, k_ctx, v_ctx, sees, scale):
    """One request in float64: q (T, Hq, D), k_new / v_new (T, Hkv, D), k_ctx /
    v_ctx (L, Hkv, D), sees (T, T) bool.  Returns out, lse, the weighted sum of
    |v| and the largest sum |q| |k| (for the tolerances).  What is not seen has
    no influence, whatever it holds."""
    T, hq, D = q.shape
    hkv, L = k_new.shape[1], k_ctx.shape[0]
    G = hq // hkv
    out = torch.zeros((T, hq, D), dtype=torch.float64)
    absum, lse = torch.zeros_like(out), torch.full((T, hq), float("-inf"), dtype=torch.float64)
    big = 0.0
    for t in range(T):
        keep = torch.cat([torch.ones(L, dtype=torch.bool), sees[t]])
        if not keep.any():
            continue
        for h in range(hq):
            k = torch.cat([k_ctx[:, h // G], k_new[:, h // G]])[keep].double()
            v = torch.cat([v_ctx[:, h // G], v_new[:, h // G]])[keep].double()
            a = (k @ q[t, h].double()) * scale
            w = torch.softmax(a, 0)
            out[t, h], absum[t, h], lse[t, h] = w @ v, w @ v.abs(), torch.logsumexp(a, 0)
            big = max(big, float((k.abs() @ q[t, h].double().abs()).max()) * scale)
    return out, lse, absum, big


def tree_bits(parents):
    """(T, T) bool: node i sees itself and its ancestors."""
    T = len(parents)
    see = torch.zeros((T, T), dtype=torch.bool)
    for i in range(T):
        k = i
        while k >= 0:
            see[i, k] = True
            k = parents[k]
    return see


def pack_bits(sees, words, junk=None):
    """int32 words of a (T, T) bool mask; bits past T from `junk` (an int)."""
    T = sees.shape[0]
    rows = []
    for i in range(T):
        b = 0 if junk is None else (junk << T) & ((1 << (32 * words)) - 1)
        for j in range(T):
            b |= int(sees[i, j]) << j
        rows.append([((b >> (32 * w)) & 0xFFFFFFFF) for w in range(words)])
    return np.array(rows, dtype=np.uint32).reshape(T, words).view(np.int32)


def verify(parents, tokens, target, draft, accept_u, sample_u):
    """The walk over one tree with exact rational sums: (path, next token).
    target, draft float32 arrays (n, V).  Follows the definition in
    include/csgmv.h with whole numbers of 2^-44."""
    f32 = np.float32
    one = f32(2.0 ** 44)

    def fixed(p):
        return [int(x) for x in np.clip(p, f32(0), f32(1)).astype(f32) * one]

    path, cur = [0], 0
    while True:
        kids = [k for k in range(len(parents)) if k > 0 and parents[k] == cur]
        p = target[cur].astype(f32)
        r, hit, taken = p.copy(), None, set()
        if draft is not None:
            q, z = draft[cur].astype(f32), f32(1)
            for k in kids:
                if not z > 0:
                    break
                if f32(f32(accept_u[k] * q[tokens[k]]) * z) < r[tokens[k]]:
                    hit = k
                    break
                r = np.maximum((r - (z * q).astype(f32)).astype(f32), f32(0))
                z = f32(f32(sum(fixed(r))) / one)
        else:
            mass, coin = 0, int(f32(accept_u[cur]) * one)
            for k in kids:
                if tokens[k] in taken:
                    continue
                taken.add(tokens[k])
                mass += fixed(p[tokens[k]:tokens[k] + 1])[0]
                if coin < mass:
                    hit = k
                    break
        if hit is None:
            break
        path.append(hit)
        cur = hit
    w = fixed(r)
    for t in taken:
        w[t] = 0
    if sum(w) == 0:
        w = fixed(p)
    total = sum(w)
    if total == 0:
        return path, -1
    aim, run = (int(f32(sample_u) * f32(2.0 ** 31)) * total) >> 31, 0
    for v, x in enumerate(w):
        run += x
        if run > aim:
            return path, v
    raise AssertionError("unreachable")


class Pool:
    """The cache as the header describes it: host arrays of the bookkeeping,
    tokens as (layer, page, slot, head, d) arrays of 16-bit patterns."""

    def __init__(self, layers, pages, ps, heads, d, seqs, max_pages, seed=0):
        rng = np.random.default_rng(seed)
        self.ps, self.max_pages = ps, max_pages
        self.k = rng.integers(0, 1 << 16, size=(layers, pages, ps, heads, d)).astype(np.uint16)
        self.v = rng.integers(0, 1 << 16, size=(layers, pages, ps, heads, d)).astype(np.uint16)
        self.table = np.full((seqs, max_pages), -1, np.int32)
        self.lens = np.zeros(seqs, np.int32)
        self.refs = np.zeros(pages, np.int32)

    def _take(self, n):
        free = [int(p) for p in np.flatnonzero(self.refs == 0)[:n]]
        for p in free:
            self.refs[p] = 1
        return free

    def _pages(self, n):
        return -(-n // self.ps)

    def commit(self, k_new, v_new, index, count, indptr, slots=None):
        """k_new / v_new (layers, tokens, heads, d) of bits."""
        todo = []
        for b in range(len(count)):
            s = b if slots is None else int(slots[b])
            old, add = int(self.lens[s]), int(count[b])
            cow = add > 0 and old % self.ps != 0 and self.refs[self.table[s, old // self.ps]] > 1
            todo.append((b, s, old, add, cow))
        need = sum(self._pages(o + a) - self._pages(o) + c for _, _, o, a, c in todo)
        if need > int((self.refs == 0).sum()):
            return False
        fresh = self._take(need)
        for b, s, old, add, cow in todo:
            if cow:
                at, new = old // self.ps, fresh.pop(0)
                src = self.table[s, at]
                for pool in (self.k, self.v):
                    pool[:, new, :old % self.ps] = pool[:, src, :old % self.ps]
                self.refs[src] -= 1
                self.table[s, at] = new
            for i in range(self._pages(old), self._pages(old + add)):
                self.table[s, i] = fresh.pop(0)
            for j in range(add):
                row = int(indptr[b]) + (j if index is None else int(index[b][j]))
                pos = old + j
                pg = self.table[s, pos // self.ps]
                self.k[:, pg, pos % self.ps] = k_new[:, row]
                self.v[:, pg, pos % self.ps] = v_new[:, row]
            self.lens[s] = old + add
        return True

    def fork(self, parents, children):
        part = [int(self.lens[a]) % self.ps != 0 for a in parents]
        if sum(part) > int((self.refs == 0).sum()):
            return False
        fresh = self._take(sum(part))
        for a, c, has in zip(parents, children, part):
            n = int(self.lens[a])
            full = n // self.ps
            for j in range(full):
                self.table[c, j] = self.table[a, j]
                self.refs[self.table[a, j]] += 1
            if has:
                new, src = fresh.pop(0), self.table[a, full]
                self.table[c, full] = new
                for pool in (self.k, self.v):
                    pool[:, new, :n % self.ps] = pool[:, src, :n % self.ps]
            self.lens[c] = n
        return True

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            n = 0 if keep is None else int(keep[i])
            if n >= self.lens[s]:
                continue
            for j in range(self._pages(n), self._pages(int(self.lens[s]))):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = n

    def compact(self):
        live = int((self.refs > 0).sum())
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        holes = [p for p in range(live) if self.refs[p] == 0]
        to = np.arange(len(self.refs), dtype=np.int32)
        for a, z in zip(movers, holes):
            to[a] = z
            self.k[:, z], self.v[:, z] = self.k[:, a], self.v[:, a]
            self.refs[z], self.refs[a] = self.refs[a], 0
        self.table = np.where(self.table >= 0, to[np.maximum(self.table, 0)], -1).astype(np.int32)

    def tokens(self, s):
        """K and V of sequence s, in order: what the bookkeeping must keep."""
        n = int(self.lens[s])
        at = [(self.table[s, i // self.ps], i % self.ps) for i in range(n)]
        return (np.stack([self.k[:, p, t] for p, t in at]) if n else None,
                np.stack([self.v[:, p, t] for p, t in at]) if n else None)
