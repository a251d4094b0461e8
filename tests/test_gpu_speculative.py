"""The serving operators run together, as examples/speculative_decode.py does:
every token that greedy decoding keeps is the best one of a plain float64
forward pass over the whole sequence, up to the rounding of bf16.

Tolerance: a layer rounds five times to bf16 (normed input, qkv, rotated q and
k, attention, output projection) and the head twice; each is a relative error
of at most 2^-9 and about 2^-10 rms, so logits (of standard deviation near 1)
move by some sqrt(12) 2^-10 = 0.3 % of it rms, and the difference of two of
them by less than 2^-5 in every one of some thousand draws."""
import pytest
import torch

from examples.speculative_decode import Decoder, Model

pytestmark = pytest.mark.gpu


def logits64(m, tokens, adapter):
    """Logits of every position of one sequence, float64, on the CPU."""
    w = lambda t: t.double().cpu()
    n, group = len(tokens), m.hq // m.hkv
    a, b, c, end = m.offsets
    pos = torch.arange(n)
    x = w(m.emb)[tokens]
    see = torch.ones((n, n), dtype=torch.bool).tril()
    for i in range(m.layers):
        h = m.norm(x)
        qkv = h @ w(m.qkv[i])
        if adapter:
            low = (h @ w(m.lora_a[i])[adapter].T).view(n, 3, m.rank)
            for s in range(3):
                lo, hi = m.offsets[s], m.offsets[s + 1]
                qkv[:, lo:hi] += low[:, s] @ w(m.lora_b[i])[adapter, lo:hi].T
        q = m.rotate(qkv[:, a:b].reshape(n, m.hq, m.d), pos)
        k = m.rotate(qkv[:, b:c].reshape(n, m.hkv, m.d), pos).repeat_interleave(group, 1)
        v = qkv[:, c:end].reshape(n, m.hkv, m.d).repeat_interleave(group, 1)
        s = torch.einsum("qhd,khd->hqk", q, k) * m.d ** -0.5
        p = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
        x = x + torch.einsum("hqk,khd->qhd", p, v).reshape(n, -1) @ w(m.o[i])
    return m.norm(x) @ w(m.head)


def prompts_of(m, lens, seed=3):
    g = torch.Generator()
    g.manual_seed(seed)
    return [torch.randint(0, m.vocab, (n,), generator=g).tolist() for n in lens]


def best_by(m, prompt, out, adapter):
    """How far each generated token's logit is below the best one, in standard deviations."""
    z = logits64(m, prompt + out[:-1], adapter)[len(prompt) - 1:]
    return (z.max(-1).values - z.gather(1, torch.tensor(out)[:, None])[:, 0]) / z.std(-1)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (4, 4, 128)])
def test_greedy_tokens_are_the_targets_best(hq, hkv, d):
    m = Model(hq=hq, hkv=hkv, d=d)
    prompts, adapters, new = prompts_of(m, [1, 2, 17, 40, 150]), [0, 1, 2, 0, 1], [20, 33, 8, 25, 30]
    dec = Decoder(m, max_seqs=6, max_len=200)
    out = dec.generate(prompts, adapters, new)
    assert dec.cache.device_status() == 0
    assert [len(o) for o in out] == new
    assert dec.kept > dec.steps  # some drafts were right
    assert int(dec.cache.page_refs.abs().sum()) == 0 and int(dec.cache.seq_lens.sum()) == 0
    for p, o, a in zip(prompts, out, adapters):
        assert float(best_by(m, p, o, a).max()) < 2.0 ** -5


def test_a_step_at_a_time_makes_the_same_claim():
    """Without drafts every step is plain decoding."""
    m = Model()
    prompts = prompts_of(m, [5, 30])
    dec = Decoder(m, max_seqs=2, max_len=64, parents=[-1])
    out = dec.generate(prompts, [1, 2], [12, 12])
    assert dec.kept == dec.steps == 24
    for p, o, a in zip(prompts, out, [1, 2]):
        assert float(best_by(m, p, o, a).max()) < 2.0 ** -5


def test_forks_share_a_prompt_and_sampling_repeats():
    m = Model()
    prompt = prompts_of(m, [75])[0]
    runs = []
    for _ in range(2):
        dec = Decoder(m, max_seqs=8, max_len=128, temperature=0.9, seed=11)
        dec.prefill([prompt], [2], [0])
        used = int((dec.cache.page_refs > 0).sum())
        dec.fork([0], [5])
        assert int((dec.cache.page_refs > 0).sum()) == used + 1  # whole pages are shared, the one begun is copied
        runs.append(dec.generate([prompt] * 2, [2, 2], [20, 20], slots=[0, 5]))
        assert dec.cache.device_status() == 0 and int(dec.cache.page_refs.abs().sum()) == 0
    assert runs[0] == runs[1]
    assert runs[0][0] != runs[0][1]
