"""The calls between the projections, the attention and the verification run
together, as examples/speculative_decode.py does, with penalties and biases:
every token that greedy decoding keeps is the best one of a plain float64 forward
pass with the same penalties, up to the rounding of bf16.  Prompts and single
tokens that go straight into the cache are seen as those of a commit are."""
import pytest
import torch

from examples.speculative_decode import Decoder, Model
from segmented_gather_gemm_gb300 import binding as B
from tests.serving_ref import attention
from tests.step_ref import Counts, HALF, scores
from tests.test_gpu_speculative import logits64, prompts_of

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def worst(m, prompt, out, adapter, rules, bias):
    """How far below the best penalised score a kept token is, in standard
    deviations of the logits; the penalties scale their rounding by at most 1.5."""
    z = logits64(m, prompt + out[:-1], adapter)[len(prompt) - 1:]
    given, most = Counts(), 0.0
    given.add(prompt[:-1], prompt=True)
    held = [prompt[-1]]
    for i, t in enumerate(out):
        given_now = Counts()
        given_now.prompt, given_now.given = given.prompt, {v: held.count(v) for v in set(held)}
        y, _ = scores(z[i], given_now, [], *rules, bias, None)
        most = max(most, float((y.max() - y[t]) / z[i].std()))
        held.append(t)
    return most


@pytest.mark.parametrize("parents", [None, [-1]])
def test_greedy_tokens_with_penalties(parents):
    m = Model()
    prompts, adapters, new = prompts_of(m, [1, 2, 17, 90]), [0, 1, 2, 1], [24, 30, 9, 28]
    rules, bias = (1.3, 0.4, 0.2), {7: 3.0, 400: -2.0, 999: 2.5}
    kw = {} if parents is None else {"parents": parents}
    dec = Decoder(m, max_seqs=5, max_len=160, repetition=rules[0], frequency=rules[1], presence=rules[2], bias=bias, **kw)
    out = dec.generate(prompts, adapters, new)
    assert dec.cache.device_status() == 0 and dec.counts.device_status() == 0
    assert not bool(dec.counts.counts.any()) and not bool(dec.counts.num_seen.any())  # ended requests are emptied
    for p, o, a in zip(prompts, out, adapters):
        # (2^-5 is test_gpu_speculative's bound for unpenalised logits)
        assert worst(m, p, o, a, rules, sorted(bias.items())) < 1.5 * 2.0 ** -5
    # the penalties tell: with a frequency this high no token stays for long
    plain = Decoder(m, max_seqs=5, max_len=160, **kw).generate(prompts, adapters, new)
    assert plain != out


def test_penalties_do_not_depend_on_drafts():
    """A tree of drafts and single tokens give the same greedy text wherever no
    two scores are near: most of it."""
    m = Model()
    prompts = prompts_of(m, [5, 40])
    kw = dict(max_seqs=2, max_len=128, repetition=1.2, frequency=0.5)
    a = Decoder(m, **kw).generate(prompts, [1, 2], [12, 12])
    b = Decoder(m, parents=[-1], **kw).generate(prompts, [1, 2], [12, 12])
    assert [x[0] for x in a] == [x[0] for x in b]


def test_sampling_with_forks_repeats():
    m = Model()
    prompt = prompts_of(m, [50])[0]
    runs = []
    for _ in range(2):
        dec = Decoder(m, max_seqs=4, max_len=128, temperature=0.8, seed=3, presence=0.5, repetition=1.1)
        dec.prefill([prompt], [1], [0])
        dec.fork([0], [3])
        assert torch.equal(dec.counts.counts[0], dec.counts.counts[3])
        runs.append(dec.generate([prompt] * 2, [1, 1], [15, 15], slots=[0, 3]))
        assert dec.cache.device_status() == dec.counts.device_status() == 0
    assert runs[0] == runs[1]


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_appended_rows_are_attended_to(layout):
    """A prompt (with the lengths before) and then single tokens (mask of zeros),
    appended and seen, against float64 over the turned keys as they were rounded."""
    g = torch.Generator().manual_seed(0)
    lens, add, hq, hkv, d = [0, 37, 5], [20, 3, 41], 4, 2, 64
    c = B.KvCache.allocate(1, 40, 16, hkv, d, 3, 8, layout=layout)
    c.k_pages.zero_(), c.v_pages.zero_()
    rope, keys, values = B.Rope(d), [[], [], []], [[], [], []]

    def append(counts):
        ptr = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        n = sum(counts)
        q, k, v = (torch.randn((n, h, d), generator=g).to(BF).cuda() for h in (hq, hkv, hkv))
        before = torch.empty(3, dtype=torch.int32, device="cuda")
        slots, pos = B.csgmv_kv_extend(c, ptr, n, lens_before=before)
        B.csgmv_kv_append(c, 0, k, v, slots, pos, rope=rope, q=q, k_out=k)
        return ptr, q, k, v, before, pos

    def check(ptr, q, out, i):
        lo, hi = ptr.tolist()[i:i + 2]
        k, v = torch.cat(keys[i]).cpu(), torch.cat(values[i]).cpu()
        n, t = k.shape[0], hi - lo
        want, _, absum, big = attention(q[lo:hi].cpu(), k[n - t:], v[n - t:], k[:n - t], v[:n - t], torch.ones(t, t, dtype=torch.bool).tril(), d ** -0.5)
        # one rounding of the output; softmax weights in 16 bits, scores in f32 (some 2^-22 of |q| |k|)
        tol = HALF[BF] * want.abs() + absum * (2.0 ** -15 + big * 2.0 ** -20)
        assert bool(((out[lo:hi].double().cpu() - want).abs() <= tol).all())

    for counts, single in ((lens, False), (add, False), ([1, 1, 1], True), ([1, 1, 1], True)):
        ptr, q, k, v, before, _ = append(counts)
        for i in range(3):
            lo, hi = ptr.tolist()[i:i + 2]
            keys[i].append(k[lo:hi])
            values[i].append(v[lo:hi])
        out = torch.empty_like(q)
        if single:
            B.csgmv_tree_attention(q, k, v, c, 0, ptr, out, mask=torch.zeros((3, 1), dtype=torch.int32, device="cuda"))
        else:
            B.csgmv_tree_attention(q, k, v, c.with_lens(before), 0, ptr, out)
        for i in range(3):
            check(ptr, q, out, i)
    assert c.device_status() == 0
