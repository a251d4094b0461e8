"""csgmv_process_logits and the counts that it goes by, against float64 and
Python's own lists.  Tolerances: tests/step_ref.py."""
import random

import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.serving_ref import pack_bits, tree_bits
from tests.step_ref import Counts, close, distribution, scores

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
BAD_SEQ, BAD_LENS, BAD_TREE, BAD_TOKEN, BAD_VALUE = 1, 8, 16, 32, 64
NONE, NAN, INF = float("-inf"), float("nan"), float("inf")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def floats(v):
    return torch.tensor(v, dtype=F32, device="cuda")


def f32(v):
    return [float(x) for x in torch.tensor(v, dtype=F32)]


def indptr(lens):
    p = [0]
    for n in lens:
        p.append(p[-1] + n)
    return p


def pack(allowed):
    """(masks, words) int32 bits of (masks, vocab) bool."""
    m, v = allowed.shape
    bits = torch.zeros((m, -(-v // 32) * 32), dtype=torch.int64)
    bits[:, :v] = allowed.cpu().long()
    w = (bits.view(m, -1, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int().cuda()


class Batch:
    """A drawn batch: what the call takes and what the reference knows."""

    def __init__(self, vocab, T, dtype=BF, seed=0, history=60, biases=5, masks=True, branch=True, stride=0, shuffle=True):
        r, g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.vocab, self.T, self.ptr, n = vocab, T, indptr(T), sum(T)
        wide = torch.randn((n, vocab + stride), generator=g) * 4
        self.logits = wide.to(dtype).cuda()[:, :vocab]
        bs = len(T)
        self.seqs = list(range(bs + 2))
        if shuffle:
            r.shuffle(self.seqs)
        self.seqs = self.seqs[:bs]
        self.ref = [Counts() for _ in range(bs)]
        self.counts = B.TokenCounts(bs + 2, vocab)
        some = [r.randrange(vocab) for _ in range(8)]
        for prompt in (True, False):
            held = [[r.choice(some) if r.random() < 0.5 else r.randrange(vocab) for _ in range(r.randint(0, history))] for _ in T]
            for c, h in zip(self.ref, held):
                c.add(h, prompt)
            B.csgmv_count_tokens(self.counts, ints([t for h in held for t in h]), ints(indptr([len(h) for h in held])),
                                 seq_slots=ints(self.seqs), prompt=prompt)
        self.rho, self.alpha, self.beta = (f32([r.choice([n, r.uniform(a, b)]) for _ in T]) for n, a, b in (
            (1.0, 0.7, 1.5), (0.0, -0.3, 0.7), (0.0, -0.5, 1.0)))
        self.heat = f32([r.choice([0.0, 1.0, r.uniform(0.2, 2.0)]) for _ in T])
        self.bias = [sorted((r.choice(some) if r.random() < 0.5 else r.randrange(vocab), x) for x in f32([r.gauss(0, 3) for _ in range(r.randint(0, biases))]))
                     for _ in T] if biases else None
        self.parents = [[-1][:t] + [r.randrange(max(0, i - 3), i) for i in range(1, t)] for t in T]
        self.drafts = [r.choice(some) if r.random() < 0.6 else r.randrange(vocab) for _ in range(n)] if branch else None
        self.allowed = self.index = None
        if masks:
            m = max(1, n // 3)
            self.allowed = torch.rand((m, vocab), generator=g) < 0.3
            self.index = [r.choice([-1, r.randrange(m)]) for _ in range(n)]
        self.words, self.trees = (max(T) + 31) // 32, None
        self.rules = B.LogitRules(
            counts=self.counts, repetition=floats(self.rho), frequency=floats(self.alpha), presence=floats(self.beta),
            temperature=floats(self.heat), allow=None if not masks else pack(self.allowed), allow_index=None if not masks else ints(self.index),
            bias=None if not biases else (ints(indptr([len(b) for b in self.bias])), ints([v for b in self.bias for v, _ in b]),
                                          floats([x for b in self.bias for _, x in b])))

    def see(self, b):
        if self.trees is None:
            self.trees = [tree_bits(p) for p in self.parents]
        return self.trees[b]

    def call(self, out=None, softmax=True):
        mask = None
        if self.drafts is not None:
            mask = torch.cat([torch.from_numpy(pack_bits(self.see(b), self.words)) for b in range(len(self.T))]).cuda()
        return B.csgmv_process_logits(self.logits, ints(self.ptr), self.rules, out, seq_slots=ints(self.seqs), softmax=softmax,
                                      draft_tokens=None if mask is None else ints(self.drafts), mask=mask)

    def row(self, b, i, softmax=True):
        """(values, tolerance) of row i of request b"""
        t = self.ptr[b] + i
        branch = []
        if self.drafts is not None:
            branch = [self.drafts[self.ptr[b] + j] for j in self.see(b)[i].nonzero()[:, 0].tolist()]
        allowed = None if self.allowed is None or self.index[t] < 0 else self.allowed[self.index[t]]
        z, off = scores(self.logits[t].cpu(), self.ref[b], branch, self.rho[b], self.alpha[b], self.beta[b],
                        self.bias[b] if self.bias else [], allowed)
        return distribution(z, off, self.heat[b]) if softmax else (z, off)

    def check(self, out, softmax=True, skip=()):
        for b, t in enumerate(self.T):
            if b in skip:
                continue
            for i in range(t):
                close(out[self.ptr[b] + i], *self.row(b, i, softmax))
        assert self.rules.device_status() == 0 or skip


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 33, 1000, 4100, 32000, 50001, 100003])
@pytest.mark.parametrize("softmax", [True, False])
def test_rows_of_trees(dtype, vocab, softmax):
    b = Batch(vocab, [1, 5, 0, 3], dtype, seed=vocab)
    b.check(b.call(softmax=softmax), softmax)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [128256, 131072, 131073, 200000, 262144])
def test_large_vocabularies(dtype, vocab):
    b = Batch(vocab, [2, 3], dtype, seed=vocab, history=3000, biases=300)
    b.check(b.call())


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("vocab,softmax", [(40000, True), (40000, False), (39999, True), (200000, True)])
def test_more_tokens_held_than_the_list_has_room_for(dtype, vocab, softmax):
    """Most of a small vocabulary, and a good part of a large one."""
    b = Batch(vocab, [2, 1, 1], dtype, seed=vocab + softmax, history=60000, biases=2000, masks=vocab != 40000)
    b.heat[0] = 0.0
    b.rules.temperature[0] = 0.0
    b.check(b.call(softmax=softmax), softmax)
    if dtype is F32:
        want = [[b.row(i, j, softmax) for j in range(t)] for i, t in enumerate(b.T)]
        out = b.call(b.logits, softmax=softmax)
        for i, t in enumerate(b.T):
            for j in range(t):
                close(out[b.ptr[i] + j], *want[i][j])


def test_results_do_not_depend_on_the_order_of_the_list():
    """The same counts listed in another order, and many runs: the same bits."""
    b = Batch(30000, [3, 2], BF, seed=77, history=20000)
    first = b.call()
    for k in range(5):
        for s in b.seqs:
            n = int(b.counts.num_seen[s])
            b.counts.seen[s, :n] = b.counts.seen[s, :n][torch.randperm(n, device="cuda")]
        assert torch.equal(b.call(), first)


@pytest.mark.parametrize("bs", [2, 33, 300, 5000])
def test_many_requests(bs):
    """One row each and some without; enough rows that a CTA has a whole one."""
    b = Batch(640, [i % 4 != 1 for i in range(bs)], F32, seed=bs, branch=False)
    b.check(b.call())


def test_deep_branches():
    """256 nodes in a line, the same tokens again and again."""
    b = Batch(500, [256, 40], BF, seed=3, masks=False)
    b.parents = [[-1] + list(range(t - 1)) for t in b.T]
    b.check(b.call())


@pytest.mark.parametrize("part", ["counts", "branch", "bias", "masks", "nothing"])
def test_parts_alone(part):
    b = Batch(3000, [4, 2], F32, seed=11, biases=6 if part == "bias" else 0, masks=part == "masks", branch=part in ("branch", "counts"))
    if part != "counts":  # nothing counted: only what is left
        b.ref = [Counts(), Counts()]
        r = b.rules
        b.rules = B.LogitRules(repetition=r.repetition, frequency=r.frequency, presence=r.presence, temperature=r.temperature,
                               bias=r.bias, allow=r.allow, allow_index=r.allow_index)
    b.check(b.call())
    if part == "nothing":
        b.rho, b.alpha, b.beta, b.heat = [1.0] * 2, [0.0] * 2, [0.0] * 2, [1.0] * 2
        b.rules = B.LogitRules()
        b.check(b.call())


@pytest.mark.parametrize("stride", [0, 3, 8])
def test_strides_and_places(stride):
    """Rows inside wider ones, in and out, aligned and not; what is beside them stays."""
    b = Batch(1000, [3, 4], F32, seed=stride, stride=stride)
    wide = torch.full((7, 1000 + stride), 5.0, device="cuda")
    b.check(b.call(wide[:, :1000]))
    assert bool((wide[:, 1000:] == 5.0).all())
    if stride == 3:
        far = torch.full((7 * 1000 + 1,), 5.0, device="cuda")
        b.check(b.call(far[1:].view(7, 1000)))
        assert far[0] == 5.0


@pytest.mark.parametrize("softmax", [True, False])
def test_in_place(softmax):
    b = Batch(2000, [3, 1, 6], F32, seed=9)
    want = [[b.row(i, j, softmax) for j in range(t)] for i, t in enumerate(b.T)]
    out = b.call(b.logits, softmax=softmax)
    assert out.data_ptr() == b.logits.data_ptr()
    for i, t in enumerate(b.T):
        for j in range(t):
            close(out[b.ptr[i] + j], *want[i][j])


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("vocab", [40, 33333])
def test_what_is_not_finite(dtype, vocab):
    """Infinities and NaN in allowed and in masked places, rows with nothing left."""
    lowest = float(torch.finfo(dtype).min)
    n = 9
    logits = (torch.randn((n, vocab), generator=torch.Generator().manual_seed(1)) * 3).to(dtype)
    allowed = torch.ones((n, vocab), dtype=torch.bool)
    logits[0, 5] = NAN                                    # all NaN
    logits[1, 6] = INF                                    # all NaN, but the first infinity at temperature 0
    logits[2, 7], logits[2, 8] = NAN, INF                 # masked: no influence
    allowed[2, 7] = allowed[2, 8] = False
    allowed[3] = False                                    # nothing
    logits[3, 3] = NAN
    logits[4] = NONE                                      # nothing either
    logits[5] = NONE                                      # one
    logits[5, vocab - 1] = -1000.0
    logits[6] = lowest                                    # all the same
    logits[7, :30] = lowest                               # masks of the type's lowest value
    logits[8, 20], logits[8, 30] = INF, INF
    logits = logits.cuda()
    for heat in (1.0, 0.25, 0.0):
        rules = B.LogitRules(temperature=floats([heat]), allow=pack(allowed), allow_index=ints(list(range(n))))
        out = B.csgmv_process_logits(logits, ints([0, n]), rules)
        for t in range(n):
            z, off = scores(logits[t].cpu(), None, [], 1.0, 0.0, 0.0, [], allowed[t])
            close(out[t], *distribution(z, off, heat))
        assert rules.device_status() == 0
    kept = B.csgmv_process_logits(logits, ints([0, n]), rules, softmax=False)
    want = torch.where(allowed.cuda(), logits.float(), NONE)
    assert torch.equal(kept.nan_to_num(7.5, INF, NONE), want.nan_to_num(7.5, INF, NONE))


def test_ties_go_to_the_lowest():
    for vocab in (1, 5, 40000, 131072):
        logits = torch.zeros((4, vocab), dtype=BF, device="cuda")
        at = [0, vocab // 2, vocab - 1]
        for t, a in enumerate(at):
            logits[t, a:] = 2.0
        out = B.csgmv_process_logits(logits, ints([0, 4]), B.LogitRules(temperature=floats([0.0])))
        want = torch.zeros_like(out)
        for t, a in enumerate(at + [0]):
            want[t, a] = 1.0
        assert torch.equal(out, want)


def test_small_and_large_temperatures():
    logits = torch.randn((4, 1000), generator=torch.Generator().manual_seed(1)).cuda()
    heats = f32([1e-3, 1e30, 1e-38, 1e-45])
    out = B.csgmv_process_logits(logits, ints([0, 1, 2, 3, 4]), B.LogitRules(temperature=floats(heats)))
    for t in (0, 1):
        z, off = scores(logits[t].cpu(), None, [], 1.0, 0.0, 0.0, [], None)
        close(out[t], *distribution(z, off, heats[t]))
    hot = torch.nn.functional.one_hot(logits.argmax(-1), 1000).float()
    assert torch.equal(out[2:], hot[2:])


def test_biases_of_one_token_add_in_turn():
    logits = torch.zeros((1, 64), device="cuda")
    v = f32([1e8, 1.0, -1e8, 3.0])
    rules = B.LogitRules(bias=(ints([0, 4]), ints([9, 9, 9, 63]), floats(v)))
    out = B.csgmv_process_logits(logits, ints([0, 1]), rules, softmax=False)
    want = torch.zeros(64)
    want[9], want[63] = (torch.tensor(v[0]) + v[1]) + v[2], 3.0
    assert torch.equal(out[0].cpu(), want)
    ban = B.LogitRules(bias=(ints([0, 1]), ints([5]), floats([NONE])))
    out = B.csgmv_process_logits(logits, ints([0, 1]), ban)
    assert out[0, 5] == 0 and bool((out[0] > 0).sum() == 63)


def test_bad_requests_are_left_out():
    """Their rows stay, the others are as ever."""
    def run(change, status, left):
        b = Batch(300, [2, 3, 1, 2], F32, seed=21)
        change(b)
        out = torch.full((8, 300), 9.0, device="cuda")
        b.call(out)
        assert b.rules.device_status() == status
        b.check(out, skip=left)
        for k in left:
            assert bool((out[b.ptr[k]:b.ptr[k + 1]] == 9.0).all())

    for name, bad in (("repetition", 0.0), ("repetition", -1.0), ("repetition", NAN), ("repetition", INF), ("temperature", -0.5),
                      ("temperature", NAN), ("temperature", INF), ("frequency", NAN), ("presence", NAN)):
        run(lambda b: getattr(b.rules, name).__setitem__(1, bad), BAD_VALUE, [1])
    for slot in (-1, 6, 2 ** 30):
        run(lambda b: b.seqs.__setitem__(2, slot), BAD_SEQ, [2])

    def unsorted(b):
        ptr, tokens, values = b.rules.bias
        b.rules.bias[0].copy_(ints([0, 0, 0, 0, 3]))
        tokens[:3] = ints([5, 4, 9])
        b.bias = [[], [], [], []]
    run(unsorted, BAD_VALUE, [3])

    def torn(b):
        b.rules.bias[0].copy_(ints([0, 0, 0, 0, 10 ** 6]))
        b.bias = [[], [], [], []]
    run(torn, BAD_VALUE, [3])


def test_biases_out_of_order_beside_a_full_list():
    """More tokens than the list holds, and the last of many biases out of order: the
    rows stay as they are."""
    b = Batch(40000, [2, 1], BF, seed=5, history=60000, biases=2000, masks=False)
    n = int(b.rules.bias[0][2] - b.rules.bias[0][1])
    assert n > 256  # not all of them are looked at by one round of threads
    b.rules.bias[1][-1] = 0
    out = torch.full((3, 40000), 9.0, device="cuda")
    b.call(out)
    assert b.rules.device_status() == BAD_VALUE
    b.check(out, skip=[1])
    assert bool((out[2] == 9.0).all())


def test_bad_rows_and_tokens():
    b = Batch(300, [2, 3], F32, seed=22, masks=True)
    b.rules.allow_index[1], b.rules.allow_index[3] = 99, -2
    out = torch.full((5, 300), 9.0, device="cuda")
    b.call(out)
    assert b.rules.device_status() == BAD_VALUE
    for t in (0, 2, 4):
        close(out[t], *b.row(int(t >= 2), t - 2 * (t >= 2)))
    assert bool((out[[1, 3]] == 9.0).all())
    # drafted tokens and biases outside the vocabulary count for nothing
    b = Batch(300, [4], F32, seed=23, masks=False, biases=0)
    b.rules = B.LogitRules(counts=b.counts, repetition=floats(b.rho), frequency=floats(b.alpha), presence=floats(b.beta),
                           temperature=floats(b.heat), bias=(ints([0, 4]), ints([-7, 2, 300, 2 ** 30]), floats([1.0, 2.0, 3.0, 4.0])))
    b.bias = [[(2, 2.0)]]
    kept = list(b.drafts)
    b.drafts[1], b.drafts[3] = -1, 300
    out = b.call()
    assert b.rules.device_status() == BAD_TOKEN
    close(out[0], *b.row(0, 0))
    see = tree_bits(b.parents[0])
    z, off = scores(b.logits[3].cpu(), b.ref[0], [kept[j] for j in (0, 2) if see[3, j]], b.rho[0], b.alpha[0], b.beta[0], b.bias[0], None)
    close(out[3], *distribution(z, off, b.heat[0]))


def test_rows_of_no_request_stay():
    logits = torch.randn((6, 100), generator=torch.Generator().manual_seed(1)).cuda()
    out = torch.full((6, 100), 9.0, device="cuda")
    rules = B.LogitRules()
    B.csgmv_process_logits(logits, ints([1, 3, 3, 5]), rules, out)
    assert bool((out[[0, 5]] == 9.0).all())
    close(out[1:5], torch.softmax(logits[1:5].double(), -1), 2.0 ** -16)
    assert rules.device_status() == 0
    # an indptr that leaves the rows
    B.csgmv_process_logits(logits, ints([0, 3, 3, 9]), rules, out)
    assert rules.device_status() == BAD_LENS


# ------------------------------------------------------------------------------------------------ counts

def same_counts(c, refs):
    """refs: {sequence: Counts}; every other sequence is empty."""
    for s in range(c.max_seqs):
        row = refs[s].row(c.vocab_size) if s in refs else [0] * c.vocab_size
        assert c.counts[s].tolist() == row
        k = int(c.num_seen[s])
        assert sorted(c.seen[s, :k].tolist()) == [v for v, n in enumerate(row) if n]


def test_counting():
    c, refs = B.TokenCounts(5, 90), {s: Counts() for s in range(5)}
    r = random.Random(4)
    for prompt in (True, False, False):
        lens = [0, 1, 700, 3]
        seqs = [4, 0, 2, 2] if not prompt else [0, 1, 2, 4]  # a sequence may come twice
        toks = [[r.randrange(90) for _ in range(n)] for n in lens]
        B.csgmv_count_tokens(c, ints([t for l in toks for t in l]), ints(indptr(lens)), seq_slots=ints(seqs), prompt=prompt)
        for s, l in zip(seqs, toks):
            refs[s].add(l, prompt)
        same_counts(c, refs)
    assert c.device_status() == 0


def test_counting_long_prompts():
    V, lens, g = 50000, [200000, 0, 3, 70001], torch.Generator().manual_seed(2)
    tokens = (V * torch.rand(sum(lens), generator=g) ** 3).int()
    c, p = B.TokenCounts(4, V), indptr(lens)
    B.csgmv_count_tokens(c, tokens.cuda(), ints(p))
    B.csgmv_count_tokens(c, tokens.cuda(), ints(p), prompt=True)
    for s in range(4):
        want = torch.bincount(tokens[p[s]:p[s + 1]].long(), minlength=V)
        assert torch.equal(c.counts[s].cpu(), (want + (want > 0) * 2 ** 30).int())
        n = int(c.num_seen[s])
        assert torch.equal(c.seen[s, :n].cpu().long().sort().values, want.nonzero()[:, 0])
    B.csgmv_count_reset(c, ints([0, 1, 2, 3]))
    assert not bool(c.counts.any()) and not bool(c.num_seen.any())


def test_counting_accepted_paths():
    """What a verification keeps, as csgmv_kv_commit takes it."""
    c, refs = B.TokenCounts(3, 50), {s: Counts() for s in range(3)}
    tokens, ptr = [7, 8, 9, 7, 1, 2, 3, 4, 5, 6], [0, 4, 4, 10]
    path, n = [[0, 1, 3, -1], [-1, -1, -1, -1], [0, 4, -1, -1]], [3, 0, 2]
    B.csgmv_count_tokens(c, ints(tokens), ints(ptr), accept_index=ints(path), accept_len=ints(n))
    refs[0].add([7, 8, 7])
    refs[2].add([1, 5])
    same_counts(c, refs)
    B.csgmv_count_tokens(c, ints(tokens), ints(ptr), accept_len=ints([2, 0, 1]), seq_slots=ints([1, 0, 2]))
    refs[1].add([7, 8])
    refs[2].add([1])
    same_counts(c, refs)
    assert c.device_status() == 0


@pytest.mark.parametrize("ptr,seqs,lens,index,status,left", [
    ([0, 2, 4], [0, 3], None, None, BAD_SEQ, [1]), ([0, 2, 4], [-1, 1], None, None, BAD_SEQ, [0]),
    ([0, 2, 90], [0, 1], None, None, BAD_LENS, [1]), ([2, 0, 4], [0, 1], None, None, BAD_LENS, [0]),
    ([-1, 2, 4], [0, 1], None, None, BAD_LENS, [0]), ([0, 2, 4], [0, 1], [3, 1], None, BAD_LENS, [0]),
    ([0, 2, 4], [0, 1], [-1, 1], None, BAD_LENS, [0]), ([0, 2, 4], [0, 1], [2, 1], [[0, 2], [0, 0]], BAD_TREE, [0]),
    ([0, 2, 4], [0, 1], [2, 1], [[0, 1], [-1, 0]], BAD_TREE, [1]), ([0, 2, 4], [0, 1], [3, 1], [[0, 1], [0, 0]], BAD_LENS, [0])])
def test_requests_not_counted(ptr, seqs, lens, index, status, left):
    c, tokens = B.TokenCounts(3, 50), [7, 8, 9, 10]
    B.csgmv_count_tokens(c, ints(tokens), ints(ptr), accept_index=None if index is None else ints(index),
                         accept_len=None if lens is None else ints(lens), seq_slots=ints(seqs))
    refs = {}
    for b in range(2):
        if b in left:
            continue
        n = ptr[b + 1] - ptr[b] if lens is None else lens[b]
        refs[seqs[b]] = Counts()
        refs[seqs[b]].add([tokens[ptr[b] + (index[b][j] if index else j)] for j in range(n)])
    same_counts(c, refs)
    assert c.device_status() == status


def test_tokens_outside_the_vocabulary():
    c, ref = B.TokenCounts(1, 50), Counts()
    B.csgmv_count_tokens(c, ints([3, -1, 50, 2 ** 31 - 1, 3, 49]), ints([0, 6]))
    ref.add([3, 3, 49])
    same_counts(c, {0: ref})
    assert c.device_status() == BAD_TOKEN


def test_resets_and_forks():
    c, r = B.TokenCounts(6, 200), random.Random(1)
    refs = {s: Counts() for s in range(3)}
    toks = [[r.randrange(200) for _ in range(60)] for _ in range(3)]
    B.csgmv_count_tokens(c, ints(sum(toks, [])), ints([0, 60, 120, 180]))
    B.csgmv_count_tokens(c, ints(sum(toks, [])), ints([30, 90, 150, 180]), prompt=True)
    flat = sum(toks, [])
    for s in range(3):
        refs[s].add(toks[s])
        refs[s].add(flat[[30, 90, 150][s]:[90, 150, 180][s]], True)
    same_counts(c, refs)
    B.csgmv_count_fork(c, ints([0, 0, 2]), ints([3, 5, 4]))
    refs.update({3: refs[0], 5: refs[0], 4: refs[2]})
    same_counts(c, refs)
    B.csgmv_count_reset(c, ints([5, 0, 0]))
    del refs[5], refs[0]
    same_counts(c, refs)
    assert c.device_status() == 0
    # a child that is not empty, comes twice, is a parent, or is none; a parent that is none
    B.csgmv_count_fork(c, ints([1, 1, 2]), ints([4, 0, 0]))
    refs[0] = refs[1]
    same_counts(c, refs)
    assert c.device_status() == BAD_SEQ
    B.csgmv_count_fork(c, ints([1, 5, 9]), ints([5, 6, 5]))  # 5 is a parent
    same_counts(c, refs)
    B.csgmv_count_fork(c, ints([1, -1, 9]), ints([5, 5, 5]))
    refs[5] = refs[1]
    same_counts(c, refs)
    c.status.zero_()
    B.csgmv_count_reset(c, ints([6, -1]))
    same_counts(c, refs)
    assert c.device_status() == BAD_SEQ
    B.csgmv_count_reset(c, ints(list(range(6))))
    same_counts(c, {})


def test_a_captured_step_is_replayed():
    """Counting and probabilities in one graph, what it reads changed in between."""
    b = Batch(32000, [4, 2], BF, seed=31, branch=False)
    tokens, ptr = ints([3, 4, 5, 6]), ints([0, 3, 4])
    seqs = ints(b.seqs)
    out = b.call()
    bp = ints(b.ptr)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        B.csgmv_count_tokens(b.counts, tokens, ptr, seq_slots=seqs)
        B.csgmv_process_logits(b.logits, bp, b.rules, out, seq_slots=seqs)
    for k in range(3):
        tokens.copy_(ints([k, 100 + k, 3, 7]))
        b.ref[0].add([k, 100 + k, 3])
        b.ref[1].add([7])
        graph.replay()
        b.check(out)
    same_counts_of = {q: ref for q, ref in zip(b.seqs, b.ref)}
    same_counts(b.counts, same_counts_of)


def test_offsets_past_32_bits():
    """More than 2^31 logits; the last rows are right."""
    vocab, n = 262144, 8200
    logits = torch.zeros((n, vocab), dtype=BF, device="cuda")
    logits[-1, 7] = 9.0
    out = torch.empty((n, vocab), dtype=F32, device="cuda")
    B.csgmv_process_logits(logits, ints([0, n]), B.LogitRules(), out)
    z = logits[-1].double().cpu()
    close(out[-1], *distribution(z, torch.zeros_like(z), 1.0))
    assert float(out[-2].min()) == float(out[-2].max())
