"""The calls between the projections, the attention and the verification: operands,
stream and current device have to be one GPU, and of the right types and shapes,
or nothing is launched; what a call with an explicit stream allocates belongs to
that stream.  (With one GPU: handles are made to say that they are on another.)"""
import pytest
import torch

from segmented_gather_gemm_gb300 import binding as B
from tests.gpu_helpers import dev_i32
from tests.step_ref import close
from tests.test_gpu_serving_streams import PAUSE

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Calls:
    """Every call, on operands that are right."""

    def __init__(self):
        self.cache = B.KvCache.allocate(1, 8, 16, 1, 64, 2, 4)
        self.rope, self.counts = B.Rope(64), B.TokenCounts(2, 100)
        self.norm = B.Norm("rms", torch.ones(64, dtype=BF, device="cuda"))
        self.rules = B.LogitRules(counts=self.counts, temperature=torch.ones(1, device="cuda"))

    def all(self, stream=None, allocate=False):
        x = torch.zeros((2, 64), dtype=BF, device="cuda")
        q, k = torch.zeros((2, 2, 64), dtype=BF, device="cuda"), torch.zeros((2, 1, 64), dtype=BF, device="cuda")
        ptr, pos, at = dev_i32([0, 2]), dev_i32([0, 1]), torch.tensor([0, -1], device="cuda")
        logits = torch.zeros((2, 100), device="cuda")
        kw = dict(stream=stream)
        given = lambda t: {} if allocate else {"out": torch.empty_like(t)}
        ext = {} if allocate else {"slots": torch.empty_like(at), "positions": torch.empty_like(pos)}
        return [lambda: B.csgmv_add_norm(x, self.norm, **given(x), **kw), lambda: B.csgmv_rotary(self.rope, pos, q, k, **kw),
                lambda: B.csgmv_kv_extend(self.cache, ptr, 2, **ext, **kw),
                lambda: B.csgmv_kv_append(self.cache, 0, k, k, at, pos, rope=self.rope, q=q, **kw),
                lambda: B.csgmv_count_tokens(self.counts, pos, ptr, **kw), lambda: B.csgmv_count_fork(self.counts, dev_i32([0]), dev_i32([1]), **kw),
                lambda: B.csgmv_count_reset(self.counts, dev_i32([0, 1]), **kw),
                lambda: B.csgmv_process_logits(logits, ptr, self.rules, **given(logits), **kw)]

    def state(self):
        return [t.clone() for t in (self.cache.page_table, self.cache.seq_lens, self.counts.counts, self.counts.num_seen)]


def test_operands_of_another_device(monkeypatch):
    c = Calls()
    before = c.state()
    for x in (c.cache, c.rope, c.counts, c.norm, c.rules):
        x.device = 1
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in c.all():
        with pytest.raises(B.CsgmvError, match="device|cuda:1"):
            call()
    assert all(torch.equal(a, b) for a, b in zip(before, c.state()))


def test_another_current_device(monkeypatch):
    c = Calls()
    before, todo = c.state(), c.all()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in todo:
        with pytest.raises(B.CsgmvError, match="current device is cuda:1"):
            call()
    assert all(torch.equal(a, b) for a, b in zip(before, c.state()))


def test_a_stream_of_another_device():
    class Other:
        device_index, cuda_stream = 1, 0

    for call in Calls().all(Other()):
        with pytest.raises(B.CsgmvError, match="the stream is on cuda:1"):
            call()


def test_a_stream_that_is_only_a_handle():
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    c, s = Calls(), torch.cuda.Stream()
    todo = c.all(Handle(s))
    s.wait_stream(torch.cuda.current_stream())
    for call in todo:
        call()
    torch.cuda.synchronize()
    assert c.cache.device_status() == c.counts.device_status() == c.rules.device_status() == 0


def test_types_and_shapes_that_are_refused():
    c = Calls()
    x, f = torch.zeros((4, 64), dtype=BF, device="cuda"), torch.zeros((4, 64), device="cuda")
    q, k = torch.zeros((4, 2, 64), dtype=BF, device="cuda"), torch.zeros((4, 1, 64), dtype=BF, device="cuda")
    pos, at, ptr = dev_i32([0, 1, 2, 3]), torch.tensor([-1] * 4, device="cuda"), dev_i32([0, 4])
    logits, one = torch.zeros((4, 100), device="cuda"), torch.ones(1, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    bad = [
        lambda: B.Norm("other"), lambda: B.Norm("rms", w.cpu()), lambda: B.Norm("rms", w[::2]), lambda: B.Norm("rms", w[None]),
        lambda: B.Norm("layer", w, w.float()), lambda: B.Norm("layer", w, w[:32]),
        lambda: B.csgmv_add_norm(x.cpu(), c.norm), lambda: B.csgmv_add_norm(x.int(), c.norm), lambda: B.csgmv_add_norm(x[0], c.norm),
        lambda: B.csgmv_add_norm(f, c.norm), lambda: B.csgmv_add_norm(x[:, :32], c.norm), lambda: B.csgmv_add_norm(x.t(), B.Norm("rms")),
        lambda: B.csgmv_add_norm(x, c.norm, f), lambda: B.csgmv_add_norm(x, c.norm, x[:2]), lambda: B.csgmv_add_norm(f, None, residual=x),
        lambda: B.csgmv_add_norm(x, c.norm, residual=x, residual_out=f), lambda: B.csgmv_add_norm(x, c.norm, residual=f[:3]),
        lambda: B.csgmv_add_norm(x, c.norm, gate=f), lambda: B.csgmv_add_norm(x, c.norm, gate=x[:2]), lambda: B.csgmv_add_norm(x, c.norm, gate=x.cpu()),
        lambda: B.csgmv_add_norm(x, None), lambda: B.csgmv_add_norm(x, c.norm, residual_out=x.half()),
        lambda: B.Rope(64, rotary_dim=66), lambda: B.Rope(64, rotary_dim=31), lambda: B.Rope(64, freq=[1.0]),
        lambda: B.Rope(64, freq=[float("inf")] * 32), lambda: B.Rope(64, device="cpu"),
        lambda: B.csgmv_rotary(c.rope, pos.long(), q), lambda: B.csgmv_rotary(c.rope, pos[:3], q), lambda: B.csgmv_rotary(c.rope, pos, q.int()),
        lambda: B.csgmv_rotary(c.rope, pos, q[..., :32]), lambda: B.csgmv_rotary(c.rope, pos, q, k.float()),
        lambda: B.csgmv_rotary(c.rope, pos, q, q_out=q.float()), lambda: B.csgmv_rotary(c.rope, pos, q, q_out=k),
        lambda: B.csgmv_rotary(c.rope, pos, q, k_out=k), lambda: B.csgmv_rotary(c.rope, pos.cpu(), q), lambda: B.csgmv_rotary(c.rope, pos, q.transpose(1, 2)),
        lambda: B.csgmv_kv_extend(c.cache, ptr.long(), 4), lambda: B.csgmv_kv_extend(c.cache, ptr, 4, add_lens=pos),
        lambda: B.csgmv_kv_extend(c.cache, ptr, 4, slots=pos), lambda: B.csgmv_kv_extend(c.cache, ptr, 4, positions=pos[:3]),
        lambda: B.csgmv_kv_extend(c.cache, ptr, 4, lens_before=pos), lambda: B.csgmv_kv_extend(c.cache, ptr, 4, seq_slots=ptr),
        lambda: B.csgmv_kv_append(c.cache, 0, q, q, at), lambda: B.csgmv_kv_append(c.cache, 0, k.half(), k, at),
        lambda: B.csgmv_kv_append(c.cache, 0, k, k, pos), lambda: B.csgmv_kv_append(c.cache, 0, k, k, at[:3]),
        lambda: B.csgmv_kv_append(c.cache, 0, k, k, at, rope=c.rope), lambda: B.csgmv_kv_append(c.cache, 0, k, k, at, pos, rope=B.Rope(128)),
        lambda: B.csgmv_kv_append(c.cache, 0, k, k, at, q_out=q), lambda: B.csgmv_kv_append(c.cache, 0, k, k, at, k_out=q),
        lambda: B.csgmv_kv_append(c.cache, 1, k, k, at), lambda: B.csgmv_kv_append(c.cache, 0, k, k, at.cpu()),
        lambda: B.csgmv_count_tokens(c.counts, pos.long(), ptr), lambda: B.csgmv_count_tokens(c.counts, pos, ptr, accept_len=pos),
        lambda: B.csgmv_count_tokens(c.counts, pos, ptr, accept_index=pos[None]), lambda: B.csgmv_count_reset(c.counts, at),
        lambda: B.csgmv_count_fork(c.counts, pos, pos[:3]), lambda: B.csgmv_count_fork(c.counts, pos, pos),
        lambda: B.LogitRules(temperature=one.double()), lambda: B.LogitRules(temperature=one, presence=torch.ones(2, device="cuda")),
        lambda: B.LogitRules(bias=(ptr, pos, one)), lambda: B.LogitRules(allow=pos[None]), lambda: B.LogitRules(allow=pos[None], allow_index=at),
        lambda: B.LogitRules(device="cpu"),
        lambda: B.csgmv_process_logits(logits.int(), ptr, c.rules), lambda: B.csgmv_process_logits(logits[:, :99], ptr, c.rules),
        lambda: B.csgmv_process_logits(logits.cpu(), ptr, c.rules), lambda: B.csgmv_process_logits(logits, dev_i32([0, 2, 4]), c.rules),
        lambda: B.csgmv_process_logits(logits, ptr, c.rules, logits[:3]), lambda: B.csgmv_process_logits(logits, ptr, c.rules, logits.double()),
        lambda: B.csgmv_process_logits(logits.bfloat16(), ptr, c.rules, logits.half()), lambda: B.csgmv_process_logits(logits.t(), ptr, B.LogitRules()),
        lambda: B.csgmv_process_logits(logits, ptr, c.rules, mask=pos[:, None]), lambda: B.csgmv_process_logits(logits, ptr, c.rules, draft_tokens=pos),
        lambda: B.csgmv_process_logits(logits, ptr, c.rules, mask=pos, draft_tokens=pos),
        lambda: B.csgmv_process_logits(logits, ptr, B.LogitRules(allow=torch.zeros((1, 3), dtype=torch.int32, device="cuda"), allow_index=pos)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(B.CsgmvError):
            call()
            pytest.fail(f"call {i} was not refused")
    assert c.counts.device_status() == c.cache.device_status() == c.rules.device_status() == 0


def test_outputs_belong_to_the_stream():
    """The current stream, after a pause, still copies a block that went back to its
    pool; a call on another stream gets memory of that one's own meanwhile."""
    g = torch.Generator().manual_seed(0)
    n, V = 64, 4096
    logits = torch.randn((n, V), generator=g).cuda()
    x = torch.randn((n, V), generator=g).cuda()
    rules, norm, ptr = B.LogitRules(), B.Norm("rms"), dev_i32([0, n])
    cache = B.KvCache.allocate(1, 64, 16, 1, 64, 1, 64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def pending(nbytes):
        t = torch.full((nbytes,), 3, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(PAUSE)
        return t.clone()

    kept = [pending(4 * n * V)]
    probs = B.csgmv_process_logits(logits, ptr, rules, stream=s)
    kept.append(pending(4 * n * V))
    out = B.csgmv_add_norm(x, norm, stream=s)
    kept.append(pending(8 * n))
    slots, pos = B.csgmv_kv_extend(cache, ptr, n, stream=s)
    others = [torch.full((4 * n * V,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((k == 3).all()) for k in kept) and all(bool((o == 255).all()) for o in others)
    close(probs, torch.softmax(logits.double(), -1), 2.0 ** -16 * torch.softmax(logits.double(), -1))
    close(out, x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6), 2.0 ** -17 * x.double().abs())
    assert slots.tolist() == list(range(n)) and pos.tolist() == list(range(n))


def test_two_streams_at_once():
    """Calls that share what they read, on two streams: each result is its own."""
    g = torch.Generator().manual_seed(1)
    logits, x = torch.randn((200, 9000), generator=g).cuda(), torch.randn((300, 4096), generator=g).to(BF).cuda()
    q = torch.randn((500, 8, 128), generator=g).to(BF).cuda()
    pos = torch.arange(500, dtype=torch.int32, device="cuda")
    rules, norm, rope, ptr = B.LogitRules(), B.Norm("layer"), B.Rope(128), dev_i32([0, 200])
    run = lambda st: (B.csgmv_process_logits(logits, ptr, rules, stream=st), B.csgmv_add_norm(x, norm, stream=st),
                      B.csgmv_rotary(rope, pos, q, q_out=torch.empty_like(q), stream=st)[0])
    want = run(None)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [run(st) for _ in range(10) for st in (a, b)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(u, v) for u, v in zip(r, want))
