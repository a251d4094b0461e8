"""The operators of a speculative serving step, as cases with a plain form.

A step drafts a tree of tokens for each sequence, scores the tree in one pass
(attention over the paged K/V cache and the drafted tokens), verifies the drafts
against the target's probabilities, appends the accepted tokens' K/V to the
cache, and between steps forks, frees and compacts pages.  ``own`` chooses
between the plain form (elementary torch operations, 32 bits) and the
framework's calls; both work on the same state.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------ cases

def _attn(name, B, tmin, tmax, lmin, lmax, hq, hkv, d, dtype, ps, layout, causal):
    return {"name": name, "op": "attention", "B": B, "tmin": tmin, "tmax": tmax, "lmin": lmin, "lmax": lmax,
            "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "ps": ps, "layout": layout, "causal": causal}


def _verify(name, B, tmin, tmax, vocab, fan, drafts):
    return {"name": name, "op": "verify", "B": B, "tmin": tmin, "tmax": tmax, "vocab": vocab, "fan": fan,
            "drafts": drafts}


def _commit(name, B, tmin, tmax, lmin, lmax, layers, hkv, d, dtype, ps, layout, prompt):
    return {"name": name, "op": "commit", "B": B, "tmin": tmin, "tmax": tmax, "lmin": lmin, "lmax": lmax,
            "layers": layers, "hkv": hkv, "d": d, "dtype": dtype, "ps": ps, "layout": layout, "prompt": prompt}


def _pages(name, B, lmin, lmax, layers, hkv, d, dtype, ps, layout):
    return {"name": name, "op": "pages", "B": B, "lmin": lmin, "lmax": lmax, "layers": layers, "hkv": hkv, "d": d,
            "dtype": dtype, "ps": ps, "layout": layout}


def listed():
    return [
        # one user's tree of a dozen drafts over a short conversation: the latency of one layer
        _attn("attn-one-user", 1, 12, 12, 1021, 1021, 32, 8, 128, "bf16", 16, "HND", False),
        # plain decoding, one token for each of 256 requests, ragged contexts
        _attn("attn-decode", 256, 1, 1, 64, 4096, 32, 8, 128, "bf16", 16, "HND", True),
        # a batch of wide trees, where the products weigh as much as the bytes
        _attn("attn-trees", 32, 33, 64, 500, 8192, 32, 8, 128, "f16", 64, "NHD", False),
        # two long documents with small trees: few rows, a long axis to split
        _attn("attn-long", 2, 16, 17, 100003, 131072, 32, 4, 64, "bf16", 32, "HND", False),
        # one user's chain of four drafts
        _verify("verify-chain", 1, 5, 5, 32000, 1, True),
        # a batch of trees whose drafts were sampled: rejections go through the residual
        _verify("verify-sampled", 64, 9, 16, 128256, 3, True),
        # a full batch whose drafts are the draft model's best tokens
        _verify("verify-best", 256, 5, 8, 128256, 4, False),
        # accepted tokens of a few users into every layer's pages
        _commit("commit-few", 4, 5, 12, 100, 900, 32, 8, 128, "bf16", 16, "HND", False),
        # accepted tokens of a full batch
        _commit("commit-batch", 256, 9, 16, 20, 120, 32, 8, 128, "bf16", 16, "HND", False),
        # a chunk of several prompts, every token kept
        _commit("commit-prompts", 8, 100, 509, 0, 300, 16, 8, 64, "f16", 64, "NHD", True),
        # a scheduler's turn over a small pool: forks, ended sequences, compaction
        _pages("pages-small", 16, 30, 400, 4, 8, 64, "bf16", 16, "HND"),
        # the same over a pool of some gigabytes
        _pages("pages-large", 512, 40, 200, 32, 8, 128, "bf16", 16, "HND"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "verify", "commit", "pages"])
    dtype, ps, layout = rng.choice(["bf16", "f16"]), rng.choice([16, 32, 64, 128]), rng.choice(["HND", "NHD"])
    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    while True:
        if op == "attention":
            B, lmax, tmax = _log_int(rng, 1, 256), _log_int(rng, 16, 131072), _log_int(rng, 1, 64)
            c = _attn("", B, rng.randint(1, tmax), tmax, rng.randint(0, lmax), lmax, hkv * rng.choice([1, 2, 4, 5, 8]),
                      hkv, d, dtype, ps, layout, rng.random() < 0.3)
            w = work(c)
            # the plain form's padded scores are bounded too
            fits = w["bytes"] <= 2.0e9 and w["flops"] <= 8e10 and B * lmax * max(tmax * c["hq"], 2 * hkv * d) <= 6e8
        elif op == "verify":
            B, tmax = _log_int(rng, 1, 256), rng.randint(1, 16)
            c = _verify("", B, rng.randint(1, tmax), tmax, _log_int(rng, 1000, 151936), rng.randint(1, 4),
                        rng.random() < 0.5)
            fits = B * tmax * c["vocab"] <= 256 * 8 * 128256 // (2 if c["drafts"] else 1)
        elif op == "commit":
            B, tmax, lmax = _log_int(rng, 1, 256), _log_int(rng, 1, 64), _log_int(rng, 4, 2000)
            c = _commit("", B, rng.randint(1, tmax), tmax, rng.randint(0, lmax), lmax, _log_int(rng, 1, 32), hkv, d,
                        dtype, ps, layout, rng.random() < 0.3)
            fits = B * (lmax + tmax + ps) * c["layers"] * hkv * d <= 256 * 150 * 32 * 8 * 128 and \
                work(c)["bytes"] <= work(listed()[8])["bytes"]
        else:
            B, lmax = _log_int(rng, 4, 512), _log_int(rng, 16, 2000)
            c = _pages("", B, rng.randint(1, lmax), lmax, _log_int(rng, 1, 32), hkv, d, dtype, ps, layout)
            fits = B * (lmax + ps) * c["layers"] * hkv * d <= 512 * 130 * 32 * 8 * 128 and \
                work(c)["bytes"] <= work(listed()[11])["bytes"]
        if fits:
            del c["name"]
            return c


# ------------------------------------------------------------------------------------------------ inputs

def _spread(r, n, lo, hi):
    """n lengths spread evenly over [lo, hi], in the order r gives: their sum does not depend on r."""
    v = [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)] if n > 1 else [hi]
    r.shuffle(v)
    return v


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _indptr(lens):
    p = [0]
    for n in lens:
        p.append(p[-1] + n)
    return p


def _trees(r, sizes, fan):
    """Parents (local, -1 at the root, earlier than the child) of one tree a request."""
    parents = []
    for n in sizes:
        kids = [0] * n
        for i in range(n):
            if i == 0:
                parents.append(-1)
                continue
            open_ = [j for j in range(max(0, i - 2 * fan), i) if kids[j] < fan] or [i - 1]
            j = r.choice(open_)
            kids[j] += 1
            parents.append(j)
    return parents


def _pool_shape(layers, pages, hkv, ps, d, layout):
    return (layers, pages, hkv, ps, d) if layout == "HND" else (layers, pages, ps, hkv, d)


def _tables(r, lens, ps, pages, max_pages):
    """A page table of scattered pages, and the pages' reference counts."""
    free = list(range(pages))
    r.shuffle(free)
    refs, rows = [0] * pages, []
    for n in lens:
        k = -(-n // ps)
        mine = [free.pop() for _ in range(k)]
        for p in mine:
            refs[p] = 1
        rows.append(mine + [-1] * (max_pages - k))
    return rows, refs


def prepare(case, seed):
    r = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return globals()["_prepare_" + case["op"]](case, r, g)


def _randn(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _prepare_attention(c, r, g):
    dt, ps, B = _DTYPES[c["dtype"]], c["ps"], c["B"]
    lens, T = _spread(r, B, c["lmin"], c["lmax"]), _spread(r, B, c["tmin"], c["tmax"])
    max_pages = -(-c["lmax"] // ps)
    pages = sum(-(-n // ps) for n in lens) + 8
    rows, refs = _tables(r, lens, ps, pages, max_pages)
    shape = _pool_shape(1, pages, c["hkv"], ps, c["d"], c["layout"])
    N, hq, hkv, d = sum(T), c["hq"], c["hkv"], c["d"]
    # q, k and v are slices of one projection's output, as the step leaves them
    qkv = _randn(g, (N, (hq + 2 * hkv) * d), dt)
    qkv[:, :hq * d] *= 2.0
    parents = None if c["causal"] else _trees(r, T, 4)
    mask = None
    if parents is not None:
        mask, at, words = [], 0, (c["tmax"] + 31) // 32
        for n in T:
            bits = []
            for i in range(n):
                p = parents[at + i]
                b = (bits[p] if p >= 0 else 0) | (1 << i)
                bits.append(b)
                mask.append([((b >> (32 * w)) & 0xFFFFFFFF) - ((b >> (32 * w + 31) & 1) << 32) for w in range(words)])
            at += n
        mask = _i32(mask)
    return {"case": c, "k_pages": _randn(g, shape, dt), "v_pages": _randn(g, shape, dt), "page_table": _i32(rows),
            "seq_lens": _i32(lens), "page_refs": _i32(refs), "q": qkv[:, :hq * d].view(N, hq, d),
            "k_new": qkv[:, hq * d:(hq + hkv) * d].view(N, hkv, d), "v_new": qkv[:, (hq + hkv) * d:].view(N, hkv, d),
            "tree_indptr": _i32(_indptr(T)), "mask": mask}


def _prepare_verify(c, r, g):
    T = _spread(r, c["B"], c["tmin"], c["tmax"])
    parents, N, V = _trees(r, T, c["fan"]), sum(T), c["vocab"]
    logits = _randn(g, (N, V), torch.float32, 5.0)  # a few tokens hold most of the mass
    target = torch.softmax(logits, -1)
    logits += _randn(g, (N, V), torch.float32, 1.0)
    draft = torch.softmax(logits, -1)
    at = torch.tensor([a for a, n in zip(_indptr(T), T) for _ in range(n)], device="cuda")
    par = torch.tensor(parents, device="cuda")
    node = torch.where(par >= 0, at + par, at)  # whose distribution a draft came from
    rank = []  # among its siblings
    a = 0
    for n in T:
        seen = [0] * n
        for i in range(n):
            p = parents[a + i]
            rank.append(seen[p] if p >= 0 else 0)
            if p >= 0:
                seen[p] += 1
        a += n
    rank = torch.tensor(rank, device="cuda")
    if c["drafts"]:
        # siblings are independent draws from the draft's distribution
        u = torch.rand(N, generator=g, device="cuda")
        tokens = torch.empty(N, dtype=torch.int32, device="cuda")
        for lo in range(0, N, 256):
            cum = torch.cumsum(draft[node[lo:lo + 256]].double(), -1)
            tokens[lo:lo + 256] = torch.searchsorted(cum, (u[lo:lo + 256].double() * cum[:, -1])[:, None]
                                                     ).clamp_(max=V - 1)[:, 0].int()
    else:
        best = torch.topk(draft, max(c["fan"], 1) + 1, -1).indices
        tokens = best[node, rank.clamp(max=best.shape[1] - 1)].int()
    return {"case": c, "target": target, "draft": draft if c["drafts"] else None, "tokens": tokens,
            "parents": _i32(parents), "tree_indptr": _i32(_indptr(T)),
            "accept_u": torch.rand(N, generator=g, device="cuda"),
            "sample_u": torch.rand(c["B"], generator=g, device="cuda")}


def _prepare_commit(c, r, g):
    dt, ps, B = _DTYPES[c["dtype"]], c["ps"], c["B"]
    lens, T = _spread(r, B, c["lmin"], c["lmax"]), _spread(r, B, c["tmin"], c["tmax"])
    max_pages = -(-(c["lmax"] + c["tmax"]) // ps)
    pages = sum(-(-(n + t) // ps) for n, t in zip(lens, T)) + 8
    rows, refs = _tables(r, lens, ps, pages, max_pages)
    N, width = sum(T), c["tmax"]
    keep, index = [], []
    for t in T:
        k = t if c["prompt"] else r.randint(1, max(1, (2 * t) // 3))
        keep.append(k)
        index.append([0] + sorted(r.sample(range(1, t), k - 1)) + [-1] * (width - k))
    shape = _pool_shape(c["layers"], pages, c["hkv"], ps, c["d"], c["layout"])
    meta = {"page_table": _i32(rows), "seq_lens": _i32(lens), "page_refs": _i32(refs)}
    s = {"case": c, "k_pages": _randn(g, shape, dt), "v_pages": _randn(g, shape, dt),
         "k_new": _randn(g, (c["layers"], N, c["hkv"], c["d"]), dt),
         "v_new": _randn(g, (c["layers"], N, c["hkv"], c["d"]), dt),
         "accept_index": _i32(index), "accept_len": _i32(keep), "tree_indptr": _i32(_indptr(T))}
    return _with_meta(s, meta)


def _prepare_pages(c, r, g):
    dt, ps, B = _DTYPES[c["dtype"]], c["ps"], c["B"]
    lens = _spread(r, B, c["lmin"], c["lmax"])
    slots = B + B // 4
    max_pages = -(-c["lmax"] // ps)
    pages = sum(-(-n // ps) for n in lens) + slots + 8
    rows, refs = _tables(r, lens, ps, pages, max_pages)
    rows += [[-1] * max_pages for _ in range(slots - B)]
    order = list(range(B))
    r.shuffle(order)
    nf = B // 4
    parents, ended = order[:nf], order[nf:2 * nf]
    shape = _pool_shape(c["layers"], pages, c["hkv"], ps, c["d"], c["layout"])
    meta = {"page_table": _i32(rows), "seq_lens": _i32(lens + [0] * (slots - B)), "page_refs": _i32(refs)}
    # half of the ended sequences go whole, the others are cut back to a third
    keep = [0 if i % 2 else lens[s] // 3 for i, s in enumerate(ended)]
    s = {"case": c, "k_pages": _randn(g, shape, dt), "v_pages": _randn(g, shape, dt), "parents": _i32(parents),
         "children": _i32(list(range(B, B + nf))), "ended": _i32(ended), "keep": _i32(keep)}
    return _with_meta(s, meta)


def _with_meta(s, meta):
    """The cache's bookkeeping as views of one buffer, and a copy of it that a pass starts from."""
    sizes = [(k, v.shape, v.numel()) for k, v in meta.items()]
    s["meta"] = torch.cat([v.reshape(-1) for v in meta.values()])
    s["meta0"] = s["meta"].clone()
    at = 0
    for k, shape, n in sizes:
        s[k] = s["meta"][at:at + n].view(shape)
        at += n
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _cache(s):
    """The framework's handle of the state's cache, made on the state's first pass and kept with it."""
    from segmented_gather_gemm_gb300 import binding as B
    if "handle" not in s:
        s["handle"] = B.KvCache(s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["page_refs"],
                                layout=s["case"]["layout"])
    return B, s["handle"]


def _own_attention(s):
    B, cache = _cache(s)
    if "workspace" not in s:
        s["workspace"] = torch.empty(B.csgmv_tree_attention_workspace_bytes(cache, s["case"]["hq"]), dtype=torch.uint8,
                                     device="cuda")
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    B.csgmv_tree_attention(s["q"], s["k_new"], s["v_new"], cache, 0, s["tree_indptr"], out, mask=s["mask"], lse=lse,
                           workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_verify(s):
    from segmented_gather_gemm_gb300 import binding as B
    c = s["case"]
    if "tree" not in s:
        s["tree"] = B.DraftTree(s["tokens"].numel(), c["tmax"])
    t = s["tree"]
    B.csgmv_build_draft_tree(t, s["parents"], s["tree_indptr"])
    index, count, token = B.csgmv_verify_drafts(s["target"], s["tokens"], s["tree_indptr"], t, s["accept_u"],
                                                s["sample_u"], draft_probs=s["draft"])
    return {"mask": t.mask, "depth": t.depth, "accept_index": index, "accept_len": count, "next_token": token}


def _own_commit(s):
    B, cache = _cache(s)
    s["meta"].copy_(s["meta0"])
    B.csgmv_kv_commit(cache, s["k_new"], s["v_new"], s["accept_index"], s["accept_len"], s["tree_indptr"])
    return {k: s[k] for k in ("k_pages", "v_pages", "page_table", "seq_lens", "page_refs")}


def _own_pages(s):
    B, cache = _cache(s)
    s["meta"].copy_(s["meta0"])
    B.csgmv_kv_fork(cache, s["parents"], s["children"])
    B.csgmv_kv_free(cache, s["ended"], s["keep"])
    B.csgmv_kv_compact(cache)
    return {k: s[k] for k in ("k_pages", "v_pages", "page_table", "seq_lens", "page_refs")}


# ------------------------------------------------------------------------------------------------ plain forms

def _padded(indptr, width):
    """(B, width) row numbers of a ragged batch, and which of them are real."""
    j = torch.arange(width, device="cuda")
    real = j < (indptr[1:] - indptr[:-1])[:, None]
    return torch.where(real, indptr[:-1, None] + j, torch.zeros_like(j)).long(), real


def _plain_attention(s):
    c, ps, hkv, d = s["case"], s["case"]["ps"], s["case"]["hkv"], s["case"]["d"]
    G, B, T, L = c["hq"] // hkv, c["B"], c["tmax"], c["lmax"]
    rows, real = _padded(s["tree_indptr"], T)
    pos = torch.arange(L, device="cuda")
    page = s["page_table"][:, pos // ps].clamp(min=0).long()
    ctx = pos < s["seq_lens"][:, None]

    def keys(pool, new):
        pool = pool[0] if c["layout"] == "NHD" else pool[0].transpose(1, 2)
        old = pool[page, (pos % ps).expand(B, L)].float()
        both = torch.cat([old, new[rows].float()], 1)
        return torch.where(torch.cat([ctx, real], 1)[:, :, None, None], both, 0.0).permute(0, 2, 1, 3)

    q = s["q"][rows].float().view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d)
    scores = torch.matmul(q, keys(s["k_pages"], s["k_new"]).transpose(2, 3)) * d ** -0.5
    j = torch.arange(T, device="cuda")
    if s["mask"] is None:
        tree = (j[:, None] >= j)[None].expand(B, T, T)
    else:
        tree = ((s["mask"][rows][:, :, j // 32] >> (j % 32)) & 1).bool()
    seen = torch.cat([ctx[:, None].expand(B, T, L), tree & real[:, None]], 2)  # (B, T, L + T)
    seen = seen[:, None, :, None].expand(B, 1, T, G, L + T).reshape(B, 1, T * G, L + T)
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, keys(s["v_pages"], s["v_new"])) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    out = out.view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, c["hq"], d)
    lse = lse.view(B, hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, c["hq"])
    n = s["q"].shape[0]
    flat = torch.where(real, rows, n)
    res = torch.empty((n + 1, c["hq"], d), dtype=s["q"].dtype, device="cuda")
    res[flat] = out.to(res.dtype)
    res_lse = torch.empty((n + 1, c["hq"]), dtype=torch.float32, device="cuda")
    res_lse[flat] = lse
    return {"out": res[:n], "lse": res_lse[:n]}


_ONE = float(2 ** 44)  # probabilities are summed and compared in steps of 2^-44


def _fixed(p):
    return (p.clamp(0.0, 1.0) * _ONE).to(torch.int64)


def _pick(w, u):
    """First index whose running sum of the whole numbers w exceeds u times their total."""
    cum = torch.cumsum(w, -1)
    total = cum[:, -1]
    U = (u * float(2 ** 31)).to(torch.int64)
    aim = U * (total >> 31) + ((U * (total & (2 ** 31 - 1))) >> 31)
    return torch.searchsorted(cum, aim[:, None], right=True)[:, 0].clamp(max=w.shape[1] - 1)


def _plain_verify(s):
    c, B, T = s["case"], s["case"]["B"], s["case"]["tmax"]
    rows, real = _padded(s["tree_indptr"], T)
    base = s["tree_indptr"][:-1].long()
    par = torch.where(real, s["parents"][rows], -1).long()
    j = torch.arange(T, device="cuda")
    # ancestors: the closure of "is itself or its parent", by squaring
    up = ((j[:, None] == j) | (par[:, :, None] == j)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    words = (T + 31) // 32
    bits = torch.zeros((B, T, words * 32), dtype=torch.int64, device="cuda")
    bits[:, :, :T] = (up > 0) & real[:, :, None]
    packed = (bits.view(B, T, words, 32) << torch.arange(32, device="cuda")).sum(-1)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int()
    mask, depth = packed[real], (up.sum(-1).int() - 1)[real]
    token, U = s["tokens"][rows].long(), s["accept_u"][rows]
    arange_b = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.int64, device="cuda")
    going = torch.ones(B, dtype=torch.bool, device="cuda")
    count = torch.ones(B, dtype=torch.int64, device="cuda")
    index = torch.full((B, T), -1, dtype=torch.int64, device="cuda")
    index[:, 0] = 0
    left = None  # what is left of the last node's distribution after its drafts were refused
    for _ in range(T):
        kids = real & (par == cur[:, None])
        order = torch.argsort(torch.where(kids, j, T + j), 1)  # children first, by index
        row = base + cur
        p = s["target"][row]
        here = p.clone() if c["drafts"] else None
        z = torch.ones(B, device="cuda")
        hit = torch.zeros(B, dtype=torch.bool, device="cuda")
        new = cur.clone()
        mass = torch.zeros(B, dtype=torch.int64, device="cuda")
        taken = torch.zeros((B, c["vocab"]), dtype=torch.bool, device="cuda") if not c["drafts"] else None
        for k in range(min(c["fan"], T)):
            i = order[:, k]
            is_kid = kids[arange_b, i]
            x = token[arange_b, i]
            test = is_kid & ~hit & going
            if c["drafts"]:
                q = s["draft"][row]
                test = test & (z > 0)
                yes = test & ((U[arange_b, i] * q[arange_b, x]) * z < here[arange_b, x])
                no = test & ~yes
                here = torch.where(no[:, None], (here - z[:, None] * q).clamp(min=0.0), here)
                z = torch.where(no, _fixed(here).sum(-1).float() / _ONE, z)
            else:
                # one coin a node: the children take their shares of [0, 1) in order
                was = taken[arange_b, x]
                mass = mass + torch.where(test & ~was, _fixed(p[arange_b, x]), 0)
                coin = (U[arange_b, cur] * _ONE).to(torch.int64)
                yes = test & ~was & (coin < mass)
                taken[arange_b, x] |= test
            new, hit = torch.where(yes, i, new), hit | yes
        end = going & ~hit
        if c["drafts"]:
            w = _fixed(here)
        else:
            w = torch.where(taken, 0, _fixed(p))
        w = torch.where((w.sum(-1) > 0)[:, None], w, _fixed(p))
        left = w if left is None else torch.where(end[:, None], w, left)
        index[arange_b, torch.where(hit, count, 0)] = torch.where(hit, new, 0)
        count = count + hit
        cur, going = new, going & hit
    return {"mask": mask, "depth": depth, "accept_index": index.int(), "accept_len": count.int(),
            "next_token": _pick(left, s["sample_u"]).int()}


def _rows_of(pool, layout):
    """The pool as (layers, pages, page_size, heads, d)."""
    return pool if layout == "NHD" else pool.transpose(2, 3)


def _free_pages(refs):
    """Pages in the order they are given out: the free ones first, lowest first."""
    return torch.argsort((refs > 0).int(), stable=True)


def _plain_commit(s):
    c, ps, B, T = s["case"], s["case"]["ps"], s["case"]["B"], s["case"]["tmax"]
    s["meta"].copy_(s["meta0"])
    old, add = s["seq_lens"].long(), s["accept_len"].long()
    have, need = (old + ps - 1) // ps, (old + add + ps - 1) // ps
    first = torch.cumsum(need - have, 0) - (need - have)
    slot = torch.arange(s["page_table"].shape[1], device="cuda")
    fresh = (slot >= have[:, None]) & (slot < need[:, None])
    pages = s["page_refs"].numel()
    pick = _free_pages(s["page_refs"])[(first[:, None] + slot - have[:, None]).clamp(0, pages - 1)]
    s["page_table"].copy_(torch.where(fresh, pick.int(), s["page_table"]))
    refs = torch.cat([s["page_refs"], s["page_refs"].new_zeros(1)])
    refs[torch.where(fresh, pick, pages)] = 1
    s["page_refs"].copy_(refs[:-1])
    s["seq_lens"].copy_((old + add).int())
    j = torch.arange(T, device="cuda")
    real = (j < add[:, None]).reshape(-1)
    src = (s["tree_indptr"][:-1, None] + s["accept_index"]).reshape(-1)
    pos = old[:, None] + j
    page = torch.gather(s["page_table"].long(), 1, (pos // ps).clamp(max=s["page_table"].shape[1] - 1)).reshape(-1)
    off = (pos % ps).reshape(-1)
    keep = real.nonzero()[:, 0]
    src, page, off = src[keep].long(), page[keep], off[keep]
    for pool, new in ((s["k_pages"], s["k_new"]), (s["v_pages"], s["v_new"])):
        _rows_of(pool, c["layout"])[:, page, off] = new[:, src]
    return {k: s[k] for k in ("k_pages", "v_pages", "page_table", "seq_lens", "page_refs")}


def _plain_pages(s):
    c, ps = s["case"], s["case"]["ps"]
    s["meta"].copy_(s["meta0"])
    pages, table = s["page_refs"].numel(), s["page_table"].long()
    slot = torch.arange(table.shape[1], device="cuda")
    lens, refs = s["seq_lens"].long(), torch.cat([s["page_refs"], s["page_refs"].new_zeros(1)])
    # fork: whole pages are shared, a partial last page is copied to a fresh one
    par, kid = s["parents"].long(), s["children"].long()
    n = lens[par]
    part = (n % ps) > 0
    fresh = _free_pages(s["page_refs"])[(torch.cumsum(part.long(), 0) - part.long())]
    rows = table[par]
    shared = slot < (n // ps)[:, None]
    refs.index_add_(0, torch.where(shared, rows, pages).reshape(-1), shared.reshape(-1).int())
    last = torch.where(part, torch.gather(rows, 1, (n // ps).clamp(max=table.shape[1] - 1)[:, None])[:, 0], pages)
    refs[torch.where(part, fresh, pages)] = 1
    table[kid] = torch.where(shared, rows, torch.where((slot == (n // ps)[:, None]) & part[:, None], fresh[:, None], -1))
    lens[kid] = n
    row = torch.arange(ps, device="cuda")
    live = ((row < (n % ps)[:, None]) & part[:, None]).reshape(-1).nonzero()[:, 0]
    src = (last[:, None] * ps + row).reshape(-1)[live]
    dst = (fresh[:, None] * ps + row).reshape(-1)[live]
    for pool in (s["k_pages"], s["v_pages"]):
        t = _rows_of(pool, c["layout"])
        t[:, dst // ps, dst % ps] = t[:, src // ps, src % ps]
    # free: the pages past what is kept lose one reference
    end, keep = s["ended"].long(), s["keep"].long()
    rows = table[end]
    gone = (slot >= ((keep + ps - 1) // ps)[:, None]) & (rows >= 0)
    refs.index_add_(0, torch.where(gone, rows, pages).reshape(-1), -gone.reshape(-1).int())
    table[end] = torch.where(gone, -1, rows)
    lens[end] = keep
    # compact: the live pages above the live count move into the holes below it
    refs = refs[:pages]
    live = refs > 0
    idx = torch.arange(pages, device="cuda")
    total = live.sum()
    src, dst = (live & (idx >= total)).nonzero()[:, 0], (~live & (idx < total)).nonzero()[:, 0]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, dst] = pool[:, src]
    to = idx.clone()
    to[src] = dst
    table = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    moved = refs.clone()
    moved[dst] = refs[src]
    moved[src] = 0
    s["page_table"].copy_(table.int())
    s["seq_lens"].copy_(lens.int())
    s["page_refs"].copy_(moved)
    return {k: s[k] for k in ("k_pages", "v_pages", "page_table", "seq_lens", "page_refs")}


# ------------------------------------------------------------------------------------------------ work

def work(case):
    c, r = case, random.Random(0)
    if c["op"] == "attention":
        lens, T = sum(_spread(r, c["B"], c["lmin"], c["lmax"])), sum(_spread(r, c["B"], c["tmin"], c["tmax"]))
        pair = (c["lmin"] + c["lmax"]) / 2 if c["B"] > 1 else c["lmax"]
        kv = 2 * (lens + T) * c["hkv"] * c["d"] * 2
        return {"bytes": kv + 2 * T * c["hq"] * c["d"] * 2 + 4 * T * c["hq"] + 4 * lens // c["ps"],
                "flops": 4.0 * T * (pair + c["tmax"]) * c["hq"] * c["d"]}
    if c["op"] == "verify":
        T = sum(_spread(r, c["B"], c["tmin"], c["tmax"]))
        # the row that the last token is drawn from, and the draft's row beside it; single entries elsewhere
        return {"bytes": c["B"] * c["vocab"] * 4 * (2 if c["drafts"] else 1) + 32 * T, "flops": 2.0 * c["B"] * c["vocab"]}
    row = 2 * c["layers"] * c["hkv"] * c["d"] * 2  # one token's K and V in every layer
    lens = _spread(r, c["B"], c["lmin"], c["lmax"])
    if c["op"] == "commit":
        T = _spread(r, c["B"], c["tmin"], c["tmax"])
        kept = sum(t if c["prompt"] else (1 + max(1, 2 * t // 3)) / 2 for t in T)
        return {"bytes": 2 * kept * row + 4 * sum(-(-(n + t) // c["ps"]) for n, t in zip(lens, T)), "flops": 0}
    nf, ps = c["B"] // 4, c["ps"]
    mean = sum(-(-n // ps) for n in lens) / c["B"]
    pages = sum(-(-n // ps) for n in lens) + c["B"] + nf + 8
    live = c["B"] * mean + nf * (1 - 1 / ps) - nf * mean * 5 / 6
    moves = live * (1 - live / pages)  # scattered live pages that lie above the live count
    return {"bytes": 2 * (nf * (ps - 1) / 2 + moves * ps) * row + 8 * pages, "flops": 0}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(prepare(case, seed))
    if case["op"] == "verify":
        return _exact_verify(prepare(case, seed))
    return None  # copies and whole numbers only


def _exact_attention(s):
    """softmax(scale q K^T) V, one request and one head at a time."""
    c, ps = s["case"], s["case"]["ps"]
    G = c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    ptr, lens = s["tree_indptr"].tolist(), s["seq_lens"].tolist()
    for b in range(c["B"]):
        lo, hi, n = ptr[b], ptr[b + 1], lens[b]
        table = s["page_table"][b, :-(-n // ps)].long()
        t = hi - lo
        if s["mask"] is None:
            tree = torch.ones((t, t), dtype=torch.bool, device="cuda").tril()
        else:
            words = s["mask"][lo:hi].long() & 0xFFFFFFFF
            tree = torch.stack([(words[:, i // 32] >> (i % 32)) & 1 for i in range(t)], 1).bool()
        hide = torch.cat([torch.zeros((t, n), dtype=torch.bool, device="cuda"), ~tree], 1)
        for h in range(c["hkv"]):
            def all_of(pool, new):
                pages = pool[0][table]
                one = pages[:, h] if c["layout"] == "HND" else pages[:, :, h]
                return torch.cat([one.reshape(-1, c["d"])[:n], new[lo:hi, h]]).double()
            K, V = all_of(s["k_pages"], s["k_new"]), all_of(s["v_pages"], s["v_new"])
            for g in range(G):
                a = (s["q"][lo:hi, h * G + g].double() @ K.T / math.sqrt(c["d"])).masked_fill(hide, float("-inf"))
                lse[lo:hi, h * G + g] = torch.logsumexp(a, -1)
                out[lo:hi, h * G + g] = torch.softmax(a, -1) @ V
    return {"out": out, "lse": lse}


def _exact_verify(s):
    """The walk down each tree, in real numbers of 64 bits."""
    c = s["case"]
    ptr, par, tok = s["tree_indptr"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    U, S = s["accept_u"].tolist(), s["sample_u"].tolist()
    words = (c["tmax"] + 31) // 32
    mask, depth, index, count, last = [], [], [], [], []
    for b in range(c["B"]):
        lo, n = ptr[b], ptr[b + 1] - ptr[b]
        for i in range(n):
            line, k = [i], i
            while par[lo + k] >= 0:
                k = par[lo + k]
                line.append(k)
            depth.append(len(line) - 1)
            word = [0] * words
            for k in line:
                word[k // 32] |= 1 << (k % 32)
            mask.append([w - 2 ** 32 if w >= 2 ** 31 else w for w in word])
        path, cur = [0], 0
        while True:
            left = s["target"][lo + cur].double()
            first, z, nxt, share = left, 1.0, None, 0.0
            seen = set()
            for k in (k for k in range(n) if par[lo + k] == cur):
                x = tok[lo + k]
                if s["draft"] is not None:
                    q = s["draft"][lo + cur].double()
                    if z <= 0:
                        break
                    if U[lo + k] * float(q[x]) * z < float(left[x]):
                        nxt = k
                        break
                    left = (left - z * q).clamp(min=0)
                    z = float(left.sum())
                elif x not in seen:
                    seen.add(x)
                    share += float(first[x])
                    if U[lo + cur] < share:
                        nxt = k
                        break
            if nxt is None:
                break
            cur = nxt
            path.append(cur)
        if s["draft"] is None and seen:
            left = left.clone()
            left[torch.tensor(sorted(seen), device="cuda")] = 0.0
        if float(left.sum()) <= 0:
            left = first
        cum = torch.cumsum(left, 0)
        last.append(min(int((cum <= S[b] * float(cum[-1])).sum()), c["vocab"] - 1))
        count.append(len(path))
        index.append(path + [-1] * (c["tmax"] - len(path)))
    return {"mask": _i32(mask), "depth": _i32(depth), "accept_index": _i32(index), "accept_len": _i32(count),
            "next_token": _i32(last)}
