"""Penalties of drafted rows go by their own branch: a tree of drafts whose path is
the text that single tokens give, with that text's later tokens as the path's
siblings, keeps the same text.  A sibling that counted, or an ancestor that did
not, would move the scores of the very tokens that are to come."""
import pytest
import torch

from examples.speculative_decode import PARENTS, Decoder, Model
from segmented_gather_gemm_gb300 import binding as B
from tests.step_ref import Counts, scores
from tests.test_gpu_speculative import logits64, prompts_of

pytestmark = pytest.mark.gpu

RULES = dict(repetition=1.2, frequency=0.5, presence=0.3)
NEW = [20, 16]
# PARENTS' longest path, and for every other node the step of the text that it has
PATH, SIBLINGS = {1: 0, 3: 1, 6: 2, 7: 3}, {2: 1, 4: 2, 5: 3}


class Told(Decoder):
    """Drafts that are the given texts' next tokens."""

    def __init__(self, *a, texts, **kw):
        super().__init__(*a, **kw)
        self.texts, self.at, self.most = texts, [0] * len(texts), 0

    def draft(self, last):
        tokens, probs = last[:, None].repeat(1, len(self.parents)), None
        for b, s in enumerate(self.now):
            for node, ahead in {**PATH, **SIBLINGS}.items():
                tokens[b, node] = self.texts[s][min(self.at[s] + ahead, len(self.texts[s]) - 1)]
        return tokens, probs

    def step(self, last, adapters, slots):
        self.now = list(slots)
        got = super().step(last, adapters, slots)
        for s, more in zip(slots, got):
            self.at[s] += len(more)
            self.most = max(self.most, len(more))
        return got


def score(m, prompt, text, adapter):
    """The penalised float64 scores of the token after prompt + text, in standard deviations of the logits."""
    z = logits64(m, prompt + text, adapter)[-1]
    given = Counts()
    given.add(prompt[:-1], prompt=True)
    held = [prompt[-1]] + text
    given.given = {v: held.count(v) for v in set(held)}
    return scores(z, given, [], *RULES.values(), [], None)[0] / z.std()


def test_a_tree_keeps_the_text_of_single_tokens(monkeypatch):
    assert [PARENTS[i] for i in (1, 3, 6, 7)] == [0, 1, 3, 6] and [PARENTS[i] for i in (2, 4, 5)] == [0, 1, 2]
    m = Model()
    prompts, adapters = prompts_of(m, [5, 40]), [1, 2]
    kw = dict(max_seqs=2, max_len=128, **RULES)
    single = Decoder(m, parents=[-1], **kw).generate(prompts, adapters, NEW)
    told = Told(m, texts=single, **kw)
    tree = told.generate(prompts, adapters, NEW)
    assert told.cache.device_status() == told.counts.device_status() == 0
    assert told.most == 5  # a whole path was kept, and a token after it
    for p, a, x, y in zip(prompts, adapters, single, tree):
        same = next((i for i, (s, t) in enumerate(zip(x, y)) if s != t), len(x))
        assert same >= 10
        if same < len(x):  # they part at two scores that bf16's roundings cannot tell apart
            z = score(m, p, x[:same], a)
            assert float(z.max() - torch.minimum(z[x[same]], z[y[same]])) < 1.5 * 2.0 ** -5
    # with siblings counted the text is another one at once
    process = B.csgmv_process_logits
    monkeypatch.setattr(B, "csgmv_process_logits", lambda *a, mask, **k: process(*a, mask=torch.full_like(mask, -1), **k))
    wrong = Told(m, texts=single, **kw).generate(prompts, adapters, NEW)
    assert all(x[:6] != y[:6] for x, y in zip(single, wrong))
