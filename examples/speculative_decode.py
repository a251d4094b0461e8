"""Speculative decoding of a batch of requests, each with its own LoRA adapter.

A small random decoder runs the library's calls as a serving loop would:

  csgmv_build_batch_info + csgmv_qkv   the adapters' part of every layer's q, k, v
  csgmv_tree_attention                 prompts (causal) and draft trees (masked)
                                       over the paged cache
  csgmv_build_draft_tree               masks and positions of the drafted tokens
  csgmv_verify_drafts                  which of them stay, and the token after
  csgmv_kv_commit                      their keys and values into the cache
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
        self.ranks = torch.tensor([0] + [rank] * (adapters - 1), dtype=torch.int32, device=device)
        self.scalings = torch.ones(adapters, device=device)

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def rotate(self, x, positions):
        """Rotary positions; x is (tokens, heads, d)."""
        half = self.d // 2
        freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
        a = (positions.double()[:, None] * freq)[:, None, :]
        c, s = a.cos().to(x.dtype), a.sin().to(x.dtype)
        u, v = x[..., :half], x[..., half:]
        return torch.cat([u * c - v * s, u * s + v * c], -1)

    def forward(self, tokens, positions, bi, cache, indptr, mask, slots, k_new, v_new):
        """Logits of the rows; their keys and values go to k_new / v_new."""
        n = tokens.numel()
        a, b, c, end = self.offsets
        x = self.emb[tokens].float()
        out = torch.empty((n, self.hq, self.d), dtype=torch.bfloat16, device=self.device)
        lora_ws = torch.empty(B.csgmv_qkv_workspace_bytes(bi, 3), dtype=torch.uint8, device=self.device)
        attn_ws = torch.empty(B.csgmv_tree_attention_workspace_bytes(cache, self.hq), dtype=torch.uint8, device=self.device)
        for i in range(self.layers):
            h = self.norm(x).to(torch.bfloat16)
            qkv = h @ self.qkv[i]
            B.csgmv_qkv(h, self.lora_a[i], self.lora_b[i], self.offsets, 3, b - a, qkv, bi, workspace=lora_ws)
            q = self.rotate(qkv[:, a:b].float().view(n, self.hq, self.d), positions).to(torch.bfloat16)
            k_new[i] = self.rotate(qkv[:, b:c].float().view(n, self.hkv, self.d), positions).to(torch.bfloat16)
            v_new[i] = qkv[:, c:end].view(n, self.hkv, self.d)
            B.csgmv_tree_attention(q, k_new[i], v_new[i], cache, i, indptr, out, mask=mask, seq_slots=slots, workspace=attn_ws)
            x = x + (out.view(n, -1) @ self.o[i]).float()
        return (self.norm(x).to(torch.bfloat16) @ self.head).float()

    def draft_logits(self, tokens):
        return (self.norm(self.emb[tokens].float()).to(torch.bfloat16) @ self.head).float()


class Decoder:
    """Speculative decoding over a paged cache with `max_seqs` sequences."""

    def __init__(self, model, max_seqs, max_len, page_size=16, parents=PARENTS, temperature=0.0, seed=0):
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

    def prefill(self, prompts, adapters, slots):
        """All of each prompt but its last token, into the cache."""
        lens = [len(p) - 1 for p in prompts]
        if not sum(lens):
            return
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        tokens = self.ints([t for p in prompts for t in p[:-1]]).long()
        positions = torch.cat([torch.arange(n, device=self.m.device) for n in lens])
        k, v = self.new_rows(at[-1])
        indptr, slots = self.ints(at), self.ints(slots)
        self.m.forward(tokens, positions, self.batch(lens, adapters), self.cache, indptr, None, slots, k, v)
        B.csgmv_kv_commit(self.cache, k, v, None, self.ints(lens), indptr, seq_slots=slots)

    def fork(self, parents, children):
        B.csgmv_kv_fork(self.cache, self.ints(parents), self.ints(children))

    def free(self, slots):
        """Ends sequences and closes the holes that they leave in the pool."""
        B.csgmv_kv_free(self.cache, self.ints(slots))
        B.csgmv_kv_compact(self.cache)

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
        positions = self.cache.seq_lens[slots.long()].repeat_interleave(width) + tree.depth
        k, v = self.new_rows(n)
        logits = m.forward(tokens.view(-1), positions, self.batch([width] * bs, adapters), self.cache, indptr, tree.mask,
                           slots, k, v)
        if self.temperature:
            probs = torch.softmax(logits / self.temperature, -1)
            draft_probs = draft_probs.view(n, -1)
        else:
            probs = torch.nn.functional.one_hot(logits.argmax(-1), m.vocab).float()
        uniforms = torch.rand(n + bs, generator=self.rng, device=m.device)
        path, count, after = B.csgmv_verify_drafts(probs, tokens.view(-1).int(), indptr, tree, uniforms[:n], uniforms[n:],
                                                   draft_probs=draft_probs)
        B.csgmv_kv_commit(self.cache, k, v, path, count, indptr, seq_slots=slots)
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
