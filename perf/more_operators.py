"""What a decoder does between the projections and the attention, as cases with a plain form.

A layer's pass adds a block's output to the residual stream and norms it, turns
queries and keys by their positions, and puts keys and values into the paged
cache; behind the last layer the logits of every row become the distribution
that verification takes: penalties for what a sequence holds already, biases, a
grammar's mask, the temperature.  ``own`` chooses between the plain form
(elementary torch operations) and the framework's calls.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases

def _norm(name, n, D, dtype, rdtype, pre, post, gate, scale):
    return {"name": name, "op": "norm", "n": n, "D": D, "dtype": dtype, "rdtype": rdtype, "pre": pre, "post": post,
            "gate": gate, "scale": scale}


def _rotary(name, n, hq, hk, d, rot, dtype, interleaved, inverse, scaling, base, pmax):
    return {"name": name, "op": "rotary", "n": n, "hq": hq, "hk": hk, "d": d, "rot": rot, "dtype": dtype,
            "interleaved": interleaved, "inverse": inverse, "scaling": scaling, "base": base, "pmax": pmax}


def _append(name, B, tmin, tmax, lmin, lmax, layers, hq, hkv, d, rot, dtype, interleaved, scaling, ps, layout):
    return {"name": name, "op": "append", "B": B, "tmin": tmin, "tmax": tmax, "lmin": lmin, "lmax": lmax,
            "layers": layers, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "dtype": dtype, "interleaved": interleaved,
            "scaling": scaling, "ps": ps, "layout": layout}


def _logits(name, B, tmin, tmax, vocab, dtype, history, bias, grammar, greedy, softmax, fresh):
    return {"name": name, "op": "logits", "B": B, "tmin": tmin, "tmax": tmax, "vocab": vocab, "dtype": dtype,
            "history": history, "bias": bias, "grammar": grammar, "greedy": greedy, "softmax": softmax, "fresh": fresh}


def listed():
    return [
        # one user's token between two blocks: the latency of one layer
        _norm("norm-one-token", 1, 4096, "bf16", "bf16", "rms", "none", "none", 1.0),
        # a decoding batch of a model that norms behind its blocks too, with a gate for each token
        _norm("norm-sandwich", 2051, 4096, "f16", "f16", "rms", "rms", "token", 0.7),
        # a full prefill, the residual stream in 32 bits
        _norm("norm-prefill", 35507, 4096, "bf16", "f32", "rms", "none", "none", 1.0),
        # the drafted tokens of one user, deep in a long document
        _rotary("rotary-tree", 12, 32, 8, 128, 128, "bf16", False, False, "wavelength", 500000.0, 131072),
        # the gradient of a partly rotated projection in 32 bits, pairs side by side
        _rotary("rotary-gradient", 4099, 16, 4, 96, 64, "f32", True, True, "linear", 10000.0, 16384),
        # a full prefill
        _rotary("rotary-prefill", 35507, 32, 8, 128, 128, "bf16", False, False, "none", 10000.0, 8192),
        # one user's next token
        _append("append-one-token", 1, 1, 1, 1021, 1021, 1, 32, 8, 128, 128, "bf16", False, "none", 16, "HND"),
        # a decoding batch, four layers
        _append("append-decode", 256, 1, 1, 64, 4096, 4, 32, 8, 128, 128, "bf16", False, "wavelength", 16, "HND"),
        # a chunk of several prompts, part of them continued, two layers
        _append("append-prompts", 16, 501, 3970, 0, 900, 2, 32, 8, 128, 128, "f16", False, "yarn", 64, "NHD"),
        # one user's chain of four drafts
        _logits("logits-chain", 1, 5, 5, 32000, "bf16", 300, 8, 0.0, 0.0, True, False),
        # requests that join a batch: what they hold is counted, then their first logits are taken
        _logits("logits-joining", 256, 1, 1, 100003, "f32", 1500, 0, 0.1, 0.5, True, True),
        # a batch of drafted trees, with biases and some grammars
        _logits("logits-trees", 64, 9, 16, 128256, "bf16", 2000, 16, 0.25, 0.1, True, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rotary", "append", "logits"])
    half = rng.choice(["bf16", "f16"])
    scaling = rng.choice(["none", "linear", "ntk", "wavelength", "yarn"])
    while True:
        if op == "norm":
            dtype = rng.choice(["bf16", "f16", "f32"])
            D = rng.choice([_log_int(rng, 32, 16384), 8 * _log_int(rng, 8, 2048), 8 * _log_int(rng, 8, 2048)])
            c = _norm("", _log_int(rng, 1, 40000), D, dtype, rng.choice([dtype, "f32"]), rng.choice(["rms", "layer"]),
                      rng.choice(["none", "rms", "layer"]), rng.choice(["none", "column", "token"]),
                      rng.choice([1.0, round(rng.uniform(0.1, 1.0), 3)]))
            most = listed()[2]
        elif op == "rotary":
            d = rng.choice([64, 80, 96, 128, 128, 192, 256])
            hk = rng.choice([1, 2, 4, 8])
            c = _rotary("", _log_int(rng, 1, 40000), hk * rng.choice([1, 2, 4, 5, 8]), hk, d,
                        rng.choice([d, d, d // 2, d // 4]), rng.choice([half, half, "f32"]), rng.random() < 0.5,
                        rng.random() < 0.3, scaling, rng.choice([10000.0, 500000.0]), _log_int(rng, 16, 1 << 20))
            most = listed()[5]
        elif op == "append":
            d = rng.choice([64, 128, 128, 80, 96])
            hkv, B, tmax = rng.choice([1, 2, 4, 8]), _log_int(rng, 1, 256), _log_int(rng, 1, 4000)
            lmax = _log_int(rng, 1, 8000)
            c = _append("", B, rng.randint(1, tmax), tmax, rng.randint(0, lmax), lmax, rng.randint(1, 4),
                        hkv * rng.choice([1, 2, 4, 5, 8]), hkv, d, rng.choice([d, d, d // 2]), half,
                        rng.random() < 0.5, scaling, rng.choice([16, 32, 64, 128]), rng.choice(["HND", "NHD"]))
            most = listed()[8]
            if B * (lmax + tmax + 256) * c["layers"] * hkv * d > 16 * 5000 * 2 * 8 * 128:
                continue
        else:
            tmax = rng.choice([1, rng.randint(1, 16)])
            c = _logits("", _log_int(rng, 1, 256), rng.randint(1, tmax), tmax, _log_int(rng, 1000, 200000),
                        rng.choice([half, half, "f32"]), _log_int(rng, 1, 4000), rng.choice([0, rng.randint(1, 300)]),
                        rng.choice([0.0, round(rng.random(), 2)]), rng.choice([0.0, round(rng.random(), 2)]),
                        rng.random() < 0.8, rng.random() < 0.3)
            most = listed()[11]
            if c["B"] * c["vocab"] > 256 * 128256:
                continue
        if work(c)["bytes"] <= work(most)["bytes"]:
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


def _randn(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def prepare(case, seed):
    r = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return globals()["_prepare_" + case["op"]](case, r, g)


def _prepare_norm(c, r, g):
    n, D, dt = c["n"], c["D"], _DTYPES[c["dtype"]]
    rdt = _DTYPES[c["rdtype"]]

    def side(kind):
        """A norm's weight and, for one that centres, its bias."""
        if kind == "none":
            return None, None
        return 1 + _randn(g, (D,), dt, 0.1), _randn(g, (D,), dt, 0.1) if kind == "layer" else None

    s = {"case": c, "x": _randn(g, (n, D), dt), "residual": _randn(g, (n, D), rdt, 2.0), "gate": None}
    s["residual"][:, ::97] *= 8.0  # a few channels stand out
    s["pre_w"], s["pre_b"] = side(c["pre"])
    s["post_w"], s["post_b"] = side(c["post"])
    if c["gate"] != "none":
        s["gate"] = _randn(g, (n if c["gate"] == "token" else 1, D), dt, 0.5)
    return s


def _prepare_rotary(c, r, g):
    n, hq, hk, d, dt = c["n"], c["hq"], c["hk"], c["d"], _DTYPES[c["dtype"]]
    # q and k are slices of one projection's output; sequences of some hundred rows begin anywhere
    qkv = _randn(g, (n, (hq + 2 * hk) * d), dt)
    pos, at = [], 0
    while at < n:
        m = min(n - at, r.randint(1, 800))
        first = r.randint(0, max(0, c["pmax"] - m))
        pos += range(first, first + m)
        at += m
    return {"case": c, "q": qkv[:, :hq * d].view(n, hq, d), "k": qkv[:, hq * d:(hq + hk) * d].view(n, hk, d),
            "positions": _i32(pos)}


def _prepare_append(c, r, g):
    dt, ps, B, d = _DTYPES[c["dtype"]], c["ps"], c["B"], c["d"]
    lens, T = _spread(r, B, c["lmin"], c["lmax"]), _spread(r, B, c["tmin"], c["tmax"])
    max_pages = -(-(c["lmax"] + c["tmax"]) // ps)
    pages = sum(-(-(n + t) // ps) for n, t in zip(lens, T)) + 8
    free = list(range(pages))
    r.shuffle(free)
    refs, rows = [0] * pages, []
    for n in lens:
        mine = [free.pop() for _ in range(-(-n // ps))]
        for p in mine:
            refs[p] = 1
        rows.append(mine + [-1] * (max_pages - len(mine)))
    shape = (c["layers"], pages, c["hkv"], ps, d) if c["layout"] == "HND" else (c["layers"], pages, ps, c["hkv"], d)
    N, hq, hkv = sum(T), c["hq"], c["hkv"]
    s = {"case": c, "k_pages": _randn(g, shape, dt), "v_pages": _randn(g, shape, dt), "tree_indptr": _i32(_indptr(T)),
         "rows": N, "q": [], "k": [], "v": []}
    for _ in range(c["layers"]):  # each layer's projection
        qkv = _randn(g, (N, (hq + 2 * hkv) * d), dt)
        s["q"].append(qkv[:, :hq * d].view(N, hq, d))
        s["k"].append(qkv[:, hq * d:(hq + hkv) * d].view(N, hkv, d))
        s["v"].append(qkv[:, (hq + hkv) * d:].view(N, hkv, d))
    # the cache's bookkeeping as views of one buffer, and a copy of it that a pass starts from
    meta = {"page_table": _i32(rows), "seq_lens": _i32(lens), "page_refs": _i32(refs)}
    s["meta"] = torch.cat([v.reshape(-1) for v in meta.values()])
    s["meta0"] = s["meta"].clone()
    at = 0
    for k, v in meta.items():
        s[k] = s["meta"][at:at + v.numel()].view(v.shape)
        at += v.numel()
    return s


def _prepare_logits(c, r, g):
    B, V = c["B"], c["vocab"]
    T = _spread(r, B, c["tmin"], c["tmax"])
    N, ptr = sum(T), _indptr(T)
    # a tree for each request: parents, and the bits of a node and its ancestors
    mask = []
    for n in T:
        bits = []
        for i in range(n):
            bits.append((bits[r.randrange(max(0, i - 4), i)] if i else 0) | (1 << i))
            mask.append([bits[i] - ((bits[i] >> 31) << 32)])
    # what each sequence holds: frequent tokens many times; the first half is its prompt
    held = _spread(r, B, max(1, c["history"] // 4), c["history"])
    H = sum(held)
    tokens = (V * torch.rand(H, generator=g, device="cuda") ** 4).int().clamp_(max=V - 1)
    hp = _indptr(held)
    # half of the drafts repeat a token of the sequence
    u = torch.rand(N, generator=g, device="cuda")
    any_ = (V * torch.rand(N, generator=g, device="cuda")).int().clamp_(max=V - 1)
    near = torch.tensor([hp[b] + r.randrange(held[b]) for b in range(B) for _ in range(T[b])], device="cuda")
    drafts = torch.where(u < 0.5, tokens[near], any_)
    req = torch.tensor([b for b in range(B) for _ in range(T[b])], device="cuda")
    logits = _randn(g, (N, V), _DTYPES[c["dtype"]], 4.0)

    def each(lo, hi, neutral, some):
        return torch.tensor([neutral if r.random() < some else r.uniform(lo, hi) for _ in range(B)], device="cuda")

    s = {"case": c, "logits": logits, "tree_indptr": _i32(ptr), "mask": _i32(mask), "drafts": drafts, "req": req,
         "repetition": each(1.02, 1.4, 1.0, 0.3), "frequency": each(0.02, 0.5, 0.0, 0.3), "presence": each(0.1, 0.8, 0.0, 0.3),
         "temperature": torch.tensor([0.0 if i < c["greedy"] * B else r.uniform(0.5, 1.3) for i in range(B)], device="cuda"),
         "held": tokens, "bias": None, "allow": None}
    s["held_req"] = torch.tensor([b for b in range(B) for _ in range(held[b])], device="cuda")
    s["in_prompt"] = torch.tensor([j < held[b] // 2 for b in range(B) for j in range(held[b])], device="cuda")
    # the same history as the framework counts it: the prompts' rows, then the others
    cut = [n // 2 for n in held]
    s["prompt_tokens"], s["prompt_indptr"] = tokens[s["in_prompt"]].contiguous(), _i32(_indptr(cut))
    s["out_tokens"], s["out_indptr"] = tokens[~s["in_prompt"]].contiguous(), _i32(_indptr([n - k for n, k in zip(held, cut)]))
    s["all_seqs"] = _i32(list(range(B)))
    if c["bias"]:
        per = [sorted(r.sample(range(V), min(V, r.randint(0, c["bias"])))) for _ in range(B)]
        total = sum(len(p) for p in per)
        s["bias"] = (_i32(_indptr([len(p) for p in per])), _i32([t for p in per for t in p]),
                     _randn(g, (total,), torch.float32, 3.0))
    if c["grammar"]:
        # a request under a grammar has a set of allowed tokens for each of its rows
        rows = [t for b in range(B) if b < c["grammar"] * B for t in range(ptr[b], ptr[b + 1])]
        index = [-1] * N
        for i, t in enumerate(rows):
            index[t] = i
        words = (V + 31) // 32
        few = torch.randint(-2 ** 31, 2 ** 31, (3, len(rows), words), generator=g, device="cuda", dtype=torch.int64)
        s["allow"] = (few[0] & few[1] & few[2]).int().contiguous()  # one token in eight
        s["allow_index"] = _i32(index)
    s["words"] = None
    if not c["fresh"]:
        s["words"] = _count_words(s)
    return s


def _count_words(s):
    """(requests, vocab) int32: how often a sequence gave a token, plus 2^30 if its prompt has it."""
    c = s["case"]
    words = torch.zeros(c["B"] * c["vocab"], dtype=torch.int32, device="cuda")
    at = s["held_req"] * c["vocab"] + s["held"].long()
    words.index_add_(0, at, (~s["in_prompt"]).int())
    prompt = torch.zeros(words.shape, dtype=torch.bool, device="cuda")
    prompt[at[s["in_prompt"]]] = True
    return (words + prompt.int() * 2 ** 30).view(c["B"], c["vocab"])


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _binding():
    from segmented_gather_gemm_gb300 import binding
    return binding


def _scaling(c):
    """What the cases' scaled positions mean: contexts of 8192 tokens stretched fourfold or eightfold."""
    return {"none": None, "linear": ("linear", 4.0), "ntk": ("ntk", 4.0),
            "wavelength": ("wavelength", 8.0, 1.0, 4.0, 8192.0), "yarn": ("yarn", 4.0, 8192.0)}[c["scaling"]]


def _own_norm(s):
    B, c = _binding(), s["case"]
    if "norms" not in s:
        s["norms"] = tuple(None if kind == "none" else B.Norm(kind, w, b, eps=1e-5) for kind, w, b in (
            (c["pre"], s["pre_w"], s["pre_b"]), (c["post"], s["post_w"], s["post_b"])))
    pre, post = s["norms"]
    after, out = torch.empty_like(s["residual"]), torch.empty_like(s["x"])
    B.csgmv_add_norm(s["x"], pre, out, residual=s["residual"], residual_out=after, post_norm=post, gate=s["gate"],
                     residual_scale=c["scale"])
    return {"residual": after, "out": out}


def _own_rotary(s):
    B, c = _binding(), s["case"]
    if "rope" not in s:
        s["rope"] = B.Rope(c["d"], rotary_dim=c["rot"], base=c["base"], interleaved=c["interleaved"], scaling=_scaling(c))
    q, k = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda"), torch.empty(s["k"].shape, dtype=s["k"].dtype, device="cuda")
    B.csgmv_rotary(s["rope"], s["positions"], s["q"], s["k"], q_out=q, k_out=k, inverse=c["inverse"])
    return {"q": q, "k": k}


def _own_append(s):
    B, c = _binding(), s["case"]
    if "handle" not in s:
        s["handle"] = B.KvCache(s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], s["page_refs"], layout=c["layout"])
        s["rope"] = B.Rope(c["d"], rotary_dim=c["rot"], interleaved=c["interleaved"], scaling=_scaling(c))
    cache, rope = s["handle"], s["rope"]
    s["meta"].copy_(s["meta0"])
    slots, positions = B.csgmv_kv_extend(cache, s["tree_indptr"], s["rows"])
    turned = []
    for layer in range(c["layers"]):
        q = torch.empty(s["q"][layer].shape, dtype=s["q"][layer].dtype, device="cuda")
        B.csgmv_kv_append(cache, layer, s["k"][layer], s["v"][layer], slots, positions, rope=rope, q=s["q"][layer], q_out=q)
        turned.append(q)
    return {"q": turned, "slots": slots, "positions": positions,
            **{k: s[k] for k in ("k_pages", "v_pages", "page_table", "seq_lens", "page_refs")}}


def _own_logits(s):
    B, c = _binding(), s["case"]
    if "rules" not in s:
        s["counts"] = B.TokenCounts(c["B"], c["vocab"])
        s["rules"] = B.LogitRules(counts=s["counts"], repetition=s["repetition"], frequency=s["frequency"],
                                  presence=s["presence"], temperature=s["temperature"], bias=s["bias"], allow=s["allow"],
                                  allow_index=s.get("allow_index"))
        if not c["fresh"]:
            _own_count(B, s)
    if c["fresh"]:
        B.csgmv_count_reset(s["counts"], s["all_seqs"])
        _own_count(B, s)
    out = torch.empty(s["logits"].shape, dtype=torch.float32, device="cuda")
    B.csgmv_process_logits(s["logits"], s["tree_indptr"], s["rules"], out, draft_tokens=s["drafts"], mask=s["mask"],
                           softmax=c["softmax"])
    return {"out": out, "counts": s["counts"].counts} if c["fresh"] else {"out": out}


def _own_count(B, s):
    B.csgmv_count_tokens(s["counts"], s["prompt_tokens"], s["prompt_indptr"], prompt=True)
    B.csgmv_count_tokens(s["counts"], s["out_tokens"], s["out_indptr"])


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_side(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w.float()
    return v + b.float() if b is not None else v


def _plain_norm(s):
    c = s["case"]
    v = _plain_side(s["x"].float(), c["post"], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        v = v * s["gate"].float()
    after = s["residual"].float() * c["scale"] + v
    return {"residual": after.to(s["residual"].dtype), "out": _plain_side(after, c["pre"], s["pre_w"], s["pre_b"]).to(s["x"].dtype)}


def _frequencies(rot, base, scaling):
    """Radians a position of each pair (64 bits), and the factor of the rotated part."""
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    if scaling is None:
        return f, 1.0
    kind, factor = scaling[:2]
    if kind == "linear":
        return f / factor, 1.0
    if kind == "ntk":
        return (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot), 1.0
    if kind == "wavelength":
        _, _, low, high, orig = scaling
        turns = orig * f / (2 * math.pi)  # in the original context
        blend = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        return f * ((1 - blend) / factor + blend), 1.0
    orig = scaling[2]

    def pair(turns):
        return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot // 2 - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64, device="cuda") - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _turn(x, positions, c, base):
    """x (rows, heads, d) turned by its positions: angles in 64 bits, the products in 32."""
    rot = c["rot"]
    f, scale = _frequencies(rot, base, _scaling(c))
    a = (positions.double()[:, None] * f)[:, None, :]
    cos, sin = (torch.cos(a) * scale).float(), (torch.sin(a) * scale).float()
    if c.get("inverse"):
        sin = -sin
    y = x.float()
    u, v = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    pair = [u * cos - v * sin, u * sin + v * cos]
    turned = torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_rotary(s):
    c = s["case"]
    return {k: _turn(s[k], s["positions"], c, c["base"]) for k in ("q", "k")}


def _plain_append(s):
    c, ps, B = s["case"], s["case"]["ps"], s["case"]["B"]
    s["meta"].copy_(s["meta0"])
    old, add = s["seq_lens"].long(), (s["tree_indptr"][1:] - s["tree_indptr"][:-1]).long()
    have, need = (old + ps - 1) // ps, (old + add + ps - 1) // ps
    first = torch.cumsum(need - have, 0) - (need - have)
    slot, pages = torch.arange(s["page_table"].shape[1], device="cuda"), s["page_refs"].numel()
    fresh = (slot >= have[:, None]) & (slot < need[:, None])
    free = torch.argsort((s["page_refs"] > 0).int(), stable=True)  # the free pages first, lowest first
    pick = free[(first[:, None] + slot - have[:, None]).clamp(0, pages - 1)]
    s["page_table"].copy_(torch.where(fresh, pick.int(), s["page_table"]))
    refs = torch.cat([s["page_refs"], s["page_refs"].new_zeros(1)])
    refs[torch.where(fresh, pick, pages)] = 1
    s["page_refs"].copy_(refs[:-1])
    s["seq_lens"].copy_((old + add).int())
    req = torch.repeat_interleave(torch.arange(B, device="cuda"), add, output_size=s["rows"])
    pos = old[req] + torch.arange(s["rows"], device="cuda") - s["tree_indptr"][req]
    page = s["page_table"][req, pos // ps].long()
    turned = []
    for layer in range(c["layers"]):
        turned.append(_turn(s["q"][layer], pos, c, 10000.0))
        for pool, new in ((s["k_pages"], _turn(s["k"][layer], pos, c, 10000.0)), (s["v_pages"], s["v"][layer])):
            rows = pool[layer] if c["layout"] == "NHD" else pool[layer].transpose(1, 2)
            rows[page, pos % ps] = new
    return {"q": turned, "slots": page * ps + pos % ps, "positions": pos.int(),
            **{k: s[k] for k in ("k_pages", "v_pages", "page_table", "seq_lens", "page_refs")}}


def _allowed(s):
    """(rows, vocab) truth values of the grammars' bits."""
    V = s["case"]["vocab"]
    j = torch.arange(V, device="cuda")
    bits = (s["allow"][s["allow_index"].clamp(min=0).long()][:, j // 32] >> (j % 32)) & 1
    return (bits != 0) | (s["allow_index"] < 0)[:, None]


def _seen(s, words):
    """For every row and token: how often the sequence or the row's own branch gave it, and whether it is there at all."""
    c, req = s["case"], s["req"]
    count, base = words[req], s["tree_indptr"][req]
    there = count != 0
    count = count & (2 ** 30 - 1)
    row, j = ((s["mask"] >> torch.arange(32, device="cuda")) & 1).nonzero(as_tuple=True)
    at = row * c["vocab"] + s["drafts"][base[row] + j].long()
    count = count.contiguous().view(-1).index_add_(0, at, torch.ones_like(at, dtype=torch.int32)).view(count.shape)
    return count, there | (count > 0)


def _plain_logits(s):
    c, req = s["case"], s["req"]
    words = _count_words(s) if c["fresh"] else s["words"]
    count, there = _seen(s, words)
    z = s["logits"].float()
    rho = s["repetition"][req][:, None]
    z = torch.where(there, torch.where(z > 0, z / rho, z * rho), z)
    z = torch.where(there, z - s["frequency"][req][:, None] * count, z)
    z = torch.where(count > 0, z - s["presence"][req][:, None], z)
    if s["bias"] is not None:
        ptr, token, value = s["bias"]
        table = torch.zeros((c["B"], c["vocab"]), device="cuda")
        table[torch.repeat_interleave(torch.arange(c["B"], device="cuda"), ptr.diff().long()), token.long()] = value
        z = z + table[req]
    if s["allow"] is not None:
        z = torch.where(_allowed(s), z, float("-inf"))
    if c["softmax"]:
        top = z.amax(-1, keepdim=True)
        heat = s["temperature"][req][:, None]
        e = torch.exp((z - top) / torch.where(heat > 0, heat, 1.0))
        index = torch.arange(c["vocab"], device="cuda")
        best = torch.where(z == top, index, c["vocab"]).amin(-1, keepdim=True)
        z = torch.where(heat > 0, e / e.sum(-1, keepdim=True), (index == best).float())
    return {"out": z, "counts": words} if c["fresh"] else {"out": z}


# ------------------------------------------------------------------------------------------------ work

def work(case):
    c, r = case, random.Random(0)
    if c["op"] == "norm":
        n, D = c["n"], c["D"]
        gate = {"none": 0, "column": 1, "token": n}[c["gate"]]
        weights = sum({"none": 0, "rms": 1, "layer": 2}[c[k]] for k in ("pre", "post"))
        return {"bytes": 2 * n * D * (_BYTES[c["dtype"]] + _BYTES[c["rdtype"]]) + (gate + weights) * D * _BYTES[c["dtype"]],
                "flops": 10.0 * n * D}
    if c["op"] == "rotary":
        row = (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": c["n"] * (2 * row * _BYTES[c["dtype"]] + 4), "flops": 3.0 * c["n"] * (c["hq"] + c["hk"]) * c["rot"]}
    if c["op"] == "append":
        T, lens = _spread(r, c["B"], c["tmin"], c["tmax"]), _spread(r, c["B"], c["lmin"], c["lmax"])
        row = (c["hq"] + 2 * c["hkv"]) * c["d"] * 2
        pages = sum(-(-(n + t) // c["ps"]) - -(-n // c["ps"]) for n, t in zip(lens, T))
        return {"bytes": sum(T) * (2 * c["layers"] * row + 12) + 12 * pages,
                "flops": 3.0 * c["layers"] * sum(T) * (c["hq"] + c["hkv"]) * c["rot"]}
    T, V = _spread(r, c["B"], c["tmin"], c["tmax"]), c["vocab"]
    held = sum(_spread(r, c["B"], max(1, c["history"] // 4), c["history"]))
    extra = c["grammar"] * sum(T) * V / 8 + c["B"] * c["bias"] * 4
    # what is held: its tokens to count (and the whole table, which a pass gives out), or the counts of its tokens
    extra += 4 * held + (4.0 * c["B"] * V if c["fresh"] else 4 * held)
    return {"bytes": sum(T) * V * (_BYTES[c["dtype"]] + 4) + int(extra), "flops": 4.0 * sum(T) * V}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _blocks(n, row):
    """Ranges of rows that keep temporaries of some ten 64-bit copies small."""
    step = max(1, int(2e8 // max(row, 1)))
    return [slice(i, min(n, i + step)) for i in range(0, n, step)]


def _exact_norm(s):
    c = s["case"]
    after, out = (torch.empty(s["x"].shape, dtype=torch.float64, device="cuda") for _ in range(2))

    def normed(v, kind, w, b):
        if kind == "none":
            return v
        mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros((), dtype=torch.float64, device="cuda")
        y = w.double() * (v - mean) / torch.sqrt((v - mean).square().mean(-1, keepdim=True) + 1e-5)
        return y if b is None else y + b.double()

    for at in _blocks(c["n"], c["D"]):
        v = normed(s["x"][at].double(), c["post"], s["post_w"], s["post_b"])
        if s["gate"] is not None:
            v = v * (s["gate"][at] if c["gate"] == "token" else s["gate"]).double()
        after[at] = c["scale"] * s["residual"][at].double() + v
        out[at] = normed(after[at], c["pre"], s["pre_w"], s["pre_b"])
    return {"residual": after, "out": out}


def _exact_turn(x, positions, c, base):
    """Each pair as a complex number, times e^(i angle)."""
    rot = c["rot"]
    f, scale = _frequencies(rot, base, _scaling(c))
    out = x.double()
    for at in _blocks(x.shape[0], x.shape[1] * x.shape[2]):
        part = out[at]
        body = part[..., :rot]
        pairs = body.unflatten(-1, (rot // 2, 2)) if c["interleaved"] else body.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        angle = positions[at].double()[:, None] * f * (-1.0 if c.get("inverse") else 1.0)
        turned = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, scale), angle)[:, None, :]
        turned = torch.view_as_real(turned)
        part[..., :rot] = turned.flatten(-2) if c["interleaved"] else turned.transpose(-1, -2).flatten(-2)
    return out


def _exact_rotary(s):
    c = s["case"]
    return {k: _exact_turn(s[k], s["positions"], c, c["base"]) for k in ("q", "k")}


def _exact_append(s):
    """The cache as lists of tokens, one request at a time."""
    c, ps = s["case"], s["case"]["ps"]
    ptr, lens, refs = s["tree_indptr"].tolist(), s["seq_lens"].tolist(), s["page_refs"].tolist()
    table = s["page_table"].tolist()
    free = iter([p for p, n in enumerate(refs) if n == 0])
    slots, positions = [], []
    for b in range(c["B"]):
        for t in range(ptr[b], ptr[b + 1]):
            at = lens[b]
            if at % ps == 0:
                page = next(free)
                table[b][at // ps], refs[page] = page, 1
            slots.append(table[b][at // ps] * ps + at % ps)
            positions.append(at)
            lens[b] = at + 1
    pos = _i32(positions)
    slot = torch.tensor(slots, device="cuda")
    pools = {}
    for name, new in (("k_pages", "k"), ("v_pages", "v")):
        pool = s[name].double()
        for layer in range(c["layers"]):
            value = _exact_turn(s["k"][layer], pos, c, 10000.0) if new == "k" else s["v"][layer].double()
            if c["layout"] == "NHD":
                pool[layer].view(-1, c["hkv"], c["d"])[slot] = value
            else:
                pool[layer][slot // ps, :, slot % ps] = value
        pools[name] = pool
    return {"q": [_exact_turn(q, pos, c, 10000.0) for q in s["q"]], "slots": slot, "positions": pos, **pools,
            "page_table": _i32(table), "seq_lens": _i32(lens), "page_refs": _i32(refs)}


def _exact_logits(s):
    """One row at a time: the row's own list of tokens, then the formula."""
    c, V = s["case"], s["case"]["vocab"]
    N = s["logits"].shape[0]
    if N * V > 2e8:
        return None
    out = torch.empty((N, V), dtype=torch.float64, device="cuda")
    ptr, mask, req = s["tree_indptr"].tolist(), s["mask"][:, 0].tolist(), s["req"].tolist()
    rho, alpha, beta, heat = (s[k].tolist() for k in ("repetition", "frequency", "presence", "temperature"))
    bias = None if s["bias"] is None else [v.tolist() for v in s["bias"]]
    index = None if s["allow"] is None else s["allow_index"].tolist()
    bounds = torch.searchsorted(s["held_req"].contiguous(), torch.arange(c["B"] + 1, device="cuda")).tolist()
    for t in range(N):
        b = req[t]
        mine = slice(bounds[b], bounds[b + 1])
        given = s["held"][mine][~s["in_prompt"][mine]].long()
        branch = [ptr[b] + j for j in range(32) if (mask[t] >> j) & 1]
        count = torch.bincount(torch.cat([given, s["drafts"][branch].long()]), minlength=V)
        there = count > 0
        there[s["held"][mine].long()] = True
        z = s["logits"][t].double()
        z[there] = torch.where(z[there] > 0, z[there] / rho[b], z[there] * rho[b])
        z = z - alpha[b] * count - beta[b] * (count > 0)
        if bias is not None:
            for i in range(bias[0][b], bias[0][b + 1]):
                z[bias[1][i]] += bias[2][i]
        if index is not None and index[t] >= 0:
            words = s["allow"][index[t]].long() & 0xFFFFFFFF
            bit = (words[:, None] >> torch.arange(32, device="cuda")) & 1
            z[bit.flatten()[:V] == 0] = float("-inf")
        if c["softmax"]:
            if heat[b] > 0:
                z = torch.softmax(z / heat[b], -1)
            else:
                hot = torch.zeros_like(z)
                hot[int((z == z.max()).nonzero()[0])] = 1.0
                z = hot
        out[t] = z
    return {"out": out, "counts": _count_words(s)} if c["fresh"] else {"out": out}
