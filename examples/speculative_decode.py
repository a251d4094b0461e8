"""Speculative decoding of a batch of requests, each with its own LoRA adapter.

A small random decoder runs the library's calls as a serving loop would:

  csgmv_build_batch_info + csgmv_qkv   the adapters' part of every layer's q, k, v
  csgmv_add_norm                       a block's output into the residual stream, and
                                       the norm before the next one
  csgmv_rotary                         positions of drafted tokens
  csgmv_kv_extend + csgmv_kv_append    prompts and single tokens, turned by their
                                       positions, straight into the cache
  csgmv_tree_attention                 prompts (causal) and draft trees (masked)
                                       over the paged cache
  csgmv_build_draft_tree               masks and positions of the drafted tokens
  csgmv_process_logits                 penalties, biases, temperature: the
                                       distributions that the tokens come from
  csgmv_verify_drafts                  which drafts stay, and the token after
  csgmv_kv_commit, csgmv_count_tokens  their keys and values into the cache, the
                                       tokens into the counts of the penalties
  csgmv_kv_fork / _free / _compact     two continuations of one prompt, requests
                                       that end

The drafter is a table of likely next tokens (the embedding against the output
matrix).  With temperature 0 its best tokens are tried and the target's best
token is kept; otherwise drafts are sampled from the drafter and every kept
token is distributed as the target says.

    python examples/speculative_decode.py
"""
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from segmented_gather_gemm_gb300 import binding as B  # noqa: E402

# node 0 is the last token; two guesses for the next one, two after the first of them, ...
PARENTS = [-1, 0, 0, 1, 1, 2, 3, 6]


class Model:
    """A random decoder with `adapters` LoRA adapters on q, k and v (adapter 0
    is the bare model).  Weights are bf16, the residual stream is f32."""

    def __init__(self, layers=2, hidden=256, hq=8, hkv=2, d=64, vocab=1000, adapters=3, rank=16, seed=0, device="cuda"):
        g = torch.Generator()
        g.manual_seed(seed)

        def weight(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(device)

        self.layers, self.hidden, self.hq, self.hkv, self.d, self.vocab = layers, hidden, hq, hkv, d, vocab
        self.rank, self.device = rank, device
        self.offsets = [0, hq * d, (hq + hkv) * d, (hq + 2 * hkv) * d]
        n = self.offsets[-1]
        self.emb = weight(vocab, hidden, std=1.0)
        self.head = weight(hidden, vocab, std=hidden ** -0.5)
        self.qkv = [weight(hidden, n, std=hidden ** -0.5) for _ in range(layers)]
        self.o = [weight(hq * d, hidden, std=0.5 * (hq * d) ** -0.5) for _ in range(layers)]
        self.lora_a = [weight(adapters, 3 * rank, hidden, std=hidden ** -0.5) for _ in range(layers)]
        self.lora_b = [weight(adapters, n, rank, std=0.5 * rank ** -0.5) for _ in range(layers)]
        self.rms = B.Norm("rms", eps=1e-6)
        self.rope = B.Rope(d, device=device)
        self.ranks = torch.tensor([0] + [rank] * (adapters - 1), dtype=torch.int32, device=device)
        self.scalings = torch.ones(adapters, device=device)

    @staticmethod
    def norm(x):
        """What self.rms is, in torch."""
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def rotate(self, x, positions):
        """What self.rope is, in torch; x is (tokens, heads, d)."""
        half = self.d // 2
        freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
        a = (positions.double()[:, None] * freq)[:, None, :]
        c, s = a.cos().to(x.dtype), a.sin().to(x.dtype)
        u, v = x[..., :half], x[..., half:]
        return torch.cat([u * c - v * s, u * s + v * c], -1)

    def forward(self, tokens, positions, bi, cache, indptr, mask, slots, k_new=None, v_new=None, at=None):
        """Logits of the rows.  Their keys and values go to k_new / v_new, or, with
        at (csgmv_kv_extend's slots), straight into the cache's pages: cache then has
        the lengths that the rows' attention is to see."""
        n = tokens.numel()
        a, b, c, end = self.offsets
        block = self.emb[tokens]
        x = torch.empty((n, self.hidden), device=self.device)
        h = torch.empty((n, self.hidden), dtype=torch.bfloat16, device=self.device)
        B.csgmv_add_norm(block, self.rms, h, residual_out=x)
        out = torch.empty((n, self.hq, self.d), dtype=torch.bfloat16, device=self.device)
        lora_ws = torch.empty(B.csgmv_qkv_workspace_bytes(bi, 3), dtype=torch.uint8, device=self.device)
        attn_ws = torch.empty(B.csgmv_tree_attention_workspace_bytes(cache, self.hq), dtype=torch.uint8, device=self.device)
        for i in range(self.layers):
            qkv = h @ self.qkv[i]
            B.csgmv_qkv(h, self.lora_a[i], self.lora_b[i], self.offsets, 3, b - a, qkv, bi, workspace=lora_ws)
            q, k, v = (qkv[:, lo:hi].view(n, -1, self.d) for lo, hi in ((a, b), (b, c), (c, end)))
            if at is None:
                B.csgmv_rotary(self.rope, positions, q, k, k_out=k_new[i])
                v_new[i] = v
                k, v = k_new[i], v_new[i]
            else:
                B.csgmv_kv_append(cache, i, k, v, at, positions, rope=self.rope, q=q, k_out=k)
            B.csgmv_tree_attention(q, k, v, cache, i, indptr, out, mask=mask, seq_slots=slots, workspace=attn_ws)
            B.csgmv_add_norm(out.view(n, -1) @ self.o[i], self.rms, h, residual=x)
        return h @ self.head

    def draft_logits(self, tokens):
        return (self.norm(self.emb[tokens].float()).to(torch.bfloat16) @ self.head).float()


class Decoder:
    """Speculative decoding over a paged cache with `max_seqs` sequences.  The
    penalties and bias ({token: value}) are every request's; a sequence's given
    tokens are counted from the last one of its prompt on."""

    def __init__(self, model, max_seqs, max_len, page_size=16, parents=PARENTS, temperature=0.0, seed=0, repetition=1.0,
                 frequency=0.0, presence=0.0, bias=None):
        m = self.m = model
        pages = -(-(max_len + len(parents)) // page_size)
        self.cache = B.KvCache.allocate(m.layers, max_seqs * pages, page_size, m.hkv, m.d, max_seqs, pages, device=m.device)
        self.parents, self.temperature = parents, temperature
        depth = [0] * len(parents)
        for i, p in enumerate(parents[1:], 1):
            depth[i] = depth[p] + 1
        self.levels = [[i for i in range(1, len(parents)) if depth[i] == x] for x in range(1, max(depth) + 1)]
        self.rng = torch.Generator(device=m.device)
        self.rng.manual_seed(seed)
        self.steps = self.kept = 0
        self.penalties, self.bias = (repetition, frequency, presence), sorted((bias or {}).items())
        self.counts = None
        if self.penalties != (1.0, 0.0, 0.0):
            self.counts = B.TokenCounts(max_seqs, m.vocab, device=m.device)

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.m.device)

    def batch(self, lens, adapters):
        """The adapters' batch info for requests of `lens` rows."""
        m, n = self.m, sum(lens)
        bi = B.BatchInfo.for_batch(len(lens), n, m.ranks.numel(), m.rank)
        B.csgmv_build_batch_info(bi, self.ints(lens), self.ints(adapters), n, m.ranks, m.scalings)
        return bi

    def new_rows(self, n):
        m = self.m
        shape = (m.layers, n, m.hkv, m.d)
        return tuple(torch.empty(shape, dtype=torch.bfloat16, device=m.device) for _ in range(2))

    def rules(self, bs):
        """What a batch's logits go through."""
        each = lambda v: torch.full((bs,), v, device=self.m.device)
        kw = {"temperature": each(float(self.temperature))}
        if self.counts is not None:
            kw.update(zip(("repetition", "frequency", "presence"), map(each, self.penalties)), counts=self.counts)
        if self.bias:
            tokens, values = zip(*self.bias)
            kw["bias"] = (torch.arange(0, len(tokens) * bs + 1, len(tokens), dtype=torch.int32, device=self.m.device),
                          self.ints(tokens * bs), torch.tensor(values * bs, device=self.m.device))
        return B.LogitRules(device=self.m.device, **kw)

    def prefill(self, prompts, adapters, slots):
        """All of each prompt but its last token, into the cache."""
        lens = [len(p) - 1 for p in prompts]
        if not sum(lens):
            return
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        tokens = self.ints([t for p in prompts for t in p[:-1]])
        indptr, slots = self.ints(at), self.ints(slots)
        before = torch.empty_like(self.cache.seq_lens)
        where, positions = B.csgmv_kv_extend(self.cache, indptr, at[-1], seq_slots=slots, lens_before=before)
        # the rows see what the cache held before, and one another
        self.m.forward(tokens.long(), positions, self.batch(lens, adapters), self.cache.with_lens(before), indptr, None, slots, at=where)
        if self.counts is not None:
            B.csgmv_count_tokens(self.counts, tokens, indptr, seq_slots=slots, prompt=True)

    def fork(self, parents, children):
        B.csgmv_kv_fork(self.cache, self.ints(parents), self.ints(children))
        if self.counts is not None:
            B.csgmv_count_fork(self.counts, self.ints(parents), self.ints(children))

    def free(self, slots):
        """Ends sequences and closes the holes that they leave in the pool."""
        B.csgmv_kv_free(self.cache, self.ints(slots))
        B.csgmv_kv_compact(self.cache)
        if self.counts is not None:
            B.csgmv_count_reset(self.counts, self.ints(slots))

    def draft(self, last):
        """Draft tokens (requests, nodes) from the last tokens, and the drafter's
        distributions if it samples."""
        m, bs, width = self.m, last.numel(), len(self.parents)
        tokens = last[:, None].repeat(1, width)
        probs = torch.zeros((bs, width, m.vocab), device=m.device) if self.temperature else None
        for level in self.levels:
            for p in sorted({self.parents[i] for i in level}):
                kids = [i for i in level if self.parents[i] == p]
                logits = m.draft_logits(tokens[:, p])
                if probs is None:
                    tokens[:, kids] = logits.topk(len(kids)).indices
                else:
                    probs[:, p] = torch.softmax(logits / self.temperature, -1)
                    tokens[:, kids] = torch.multinomial(probs[:, p], len(kids), replacement=True, generator=self.rng)
        return tokens, probs

    def step(self, last, adapters, slots):
        """One target pass: the tokens that each request gains."""
        m, bs, width = self.m, len(last), len(self.parents)
        n = bs * width
        last, slots = self.ints(last).long(), self.ints(slots)
        tokens, draft_probs = self.draft(last)
        indptr = torch.arange(0, n + 1, width, dtype=torch.int32, device=m.device)
        tree = B.DraftTree(n, width, device=m.device)
        B.csgmv_build_draft_tree(tree, self.ints(self.parents * bs), indptr)
        flat, bi, k = tokens.view(-1).int(), self.batch([width] * bs, adapters), None
        if width == 1:
            # plain decoding: the token goes straight into the cache, and is seen from there
            where, positions = B.csgmv_kv_extend(self.cache, indptr, n, seq_slots=slots)
            logits = m.forward(tokens.view(-1), positions, bi, self.cache, indptr, torch.zeros_like(tree.mask), slots, at=where)
        else:
            positions = self.cache.seq_lens[slots.long()].repeat_interleave(width) + tree.depth
            k, v = self.new_rows(n)
            logits = m.forward(tokens.view(-1), positions, bi, self.cache, indptr, tree.mask, slots, k, v)
        probs = B.csgmv_process_logits(logits, indptr, self.rules(bs), draft_tokens=flat, mask=tree.mask, seq_slots=slots)
        if self.temperature:
            draft_probs = draft_probs.view(n, -1)
        uniforms = torch.rand(n + bs, generator=self.rng, device=m.device)
        path, count, after = B.csgmv_verify_drafts(probs, flat, indptr, tree, uniforms[:n], uniforms[n:], draft_probs=draft_probs)
        if k is not None:
            B.csgmv_kv_commit(self.cache, k, v, path, count, indptr, seq_slots=slots)
        if self.counts is not None:
            B.csgmv_count_tokens(self.counts, flat, indptr, path, count, seq_slots=slots)
        path, count, after, tokens = (t.tolist() for t in (path, count, after, tokens))
        self.steps += bs
        self.kept += sum(count)
        return [[tokens[b][i] for i in path[b][1:count[b]]] + [after[b]] for b in range(bs)]

    def generate(self, prompts, adapters, new_tokens, slots=None):
        """Up to new_tokens[b] tokens for each request, in slots that hold
        all of its prompt but the last token (None: 0, 1, ..., filled here)."""
        if slots is None:
            slots = list(range(len(prompts)))
            self.prefill(prompts, adapters, slots)
        out = [[] for _ in prompts]
        live = [b for b in range(len(prompts)) if new_tokens[b] > 0]
        while live:
            last = [(prompts[b] + out[b])[-1] for b in live]
            got = self.step(last, [adapters[b] for b in live], [slots[b] for b in live])
            for b, more in zip(live, got):
                out[b] += more
            done = [b for b in live if len(out[b]) >= new_tokens[b]]
            if done:
                self.free([slots[b] for b in done])
            live = [b for b in live if b not in done]
        return [o[:n] for o, n in zip(out, new_tokens)]


def main():
    model = Model()
    g = torch.Generator()
    g.manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (1, 17, 40, 130)]
    adapters, new = [0, 1, 2, 1], [48, 32, 64, 40]
    for temperature in (0.0, 0.8):
        dec = Decoder(model, max_seqs=8, max_len=256, temperature=temperature)
        t0 = time.time()
        out = dec.generate(prompts, adapters, new)
        dt = time.time() - t0
        print(f"temperature {temperature}: {sum(map(len, out))} tokens in {dt:.2f} s, {dec.kept / dec.steps:.2f} tokens kept a step")
    # two continuations of one prompt share its pages until they part
    dec = Decoder(model, max_seqs=8, max_len=256, temperature=0.8)
    dec.prefill([prompts[3]], [2], [0])
    dec.fork([0], [5])
    both = dec.generate([prompts[3]] * 2, [2, 2], [12, 12], slots=[0, 5])
    print("one prompt, two continuations:", *both)
    assert dec.cache.device_status() == 0 and int(dec.cache.page_refs.sum()) == 0


if __name__ == "__main__":
    main()
