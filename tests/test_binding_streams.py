"""Memory that a call of the binding allocates for itself when it runs on a stream of its own.

The caching allocator keeps a pool for each stream and hands a dropped block out again to the
stream whose pool it is from, whatever other streams still do with it.  On the CPU the
library, the streams and the checks are stand-ins and only the allocations are looked at; on
the GPU the other stream is held up while the current one takes every block that it can get.
"""
import contextlib

import pytest
import torch

from gated_delta_rule_spec_gb300 import binding


class FakeStream:
    cuda_stream = 77


class FakeLibrary:
    """Every call succeeds and does nothing."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name == "gdn_spec_tree_attn_workspace" else 0


class Watch:
    """The binding over stand-ins: `made` lists (shape, dtype, the stream that was current), `noted` the
    other streams that a tensor is said to be used on."""

    def __init__(self, monkeypatch):
        self.made, self.noted, self.now = [], [], None
        empty = torch.empty

        @contextlib.contextmanager
        def under(stream):
            before, self.now = self.now, stream
            yield
            self.now = before

        def make(*shape, dtype=None, device=None):
            x = empty(*shape, dtype=dtype, device="cpu")
            self.made.append((tuple(x.shape), dtype, self.now))
            return x

        monkeypatch.setattr(binding, "load", lambda lib=FakeLibrary(): lib)
        monkeypatch.setattr(binding, "_need", lambda *a: None)
        monkeypatch.setattr(binding, "_token_stride", lambda t, *a: 8)
        monkeypatch.setattr(binding, "_stream", lambda s: 5 if s is None else s.cuda_stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda: "current")
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.noted.append((tuple(t.shape), s)))
        monkeypatch.setattr(torch.cuda, "stream", under)
        monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
        self.cache = binding.KvCache(1, 4, 2, 16, 64, 2, 4, device="cpu")
        self.slots = torch.zeros(2, dtype=torch.int32)
        self.q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
        monkeypatch.setattr(torch, "empty", make)


def test_the_workspace_is_taken_where_the_call_runs(monkeypatch):
    w, s = Watch(monkeypatch), FakeStream()
    binding.tree_attn(w.cache, 0, w.slots, w.q, out=w.q, stream=s)
    assert w.made == [((4096,), torch.uint8, s)]


def results(w):
    """Calls that make what they return, as functions of the stream: (call, shapes)."""
    plan, layer = binding.RopePlan(64), binding.SpecLayer(2, 4, 32, 32, 3, 16, 2, device="cpu")
    cur = binding.SpecCursors(2, device="cpu")
    args = [w.q] * 7
    ring = layer.new_dring()
    out, snap = (2, 3, 4, 32), (2, 3, 4, 32, 32)
    return [
        (lambda s: binding.tree_attn(w.cache, 0, w.slots, w.q, workspace=w.slots, stream=s), [(2, 3, 4, 64)]),
        (lambda s: binding.rope_append(plan, w.cache, 0, w.slots, w.q, w.q, w.q, stream=s), [(2, 3, 4, 64)]),
        (lambda s: binding.rope(plan, w.slots, w.q[0], stream=s), [(3, 4, 64)]),
        (lambda s: binding.kv_reserve(w.cache, w.slots, 4, stream=s), [(2,)]),
        (lambda s: binding.kv_fork(w.cache, w.slots, w.slots, stream=s), [(2,)]),
        (lambda s: binding.verify(layer, cur, w.slots, *args, stream=s), [out]),
        (lambda s: binding.verify_d(layer, ring, cur, w.slots, *args, stream=s), [out]),
        (lambda s: binding.prefill(layer, cur, w.slots, *args, stream=s), [out]),
        (lambda s: binding.snapshot_verify(layer, cur, w.slots, *args, stream=s), [out, snap])]


@pytest.mark.parametrize("which", range(9))
def test_results_are_taken_where_the_call_runs(monkeypatch, which):
    plan = binding.RopePlan(64)
    w, s = Watch(monkeypatch), FakeStream()
    monkeypatch.setattr(binding, "RopePlan", lambda D: plan)
    call, shapes = results(w)[which]
    call(s)
    assert [(x[0], x[2]) for x in w.made] == [(shape, s) for shape in shapes]
    assert w.noted == [(shape, "current") for shape in shapes]


@pytest.mark.parametrize("which", range(9))
def test_no_stream_and_the_current_one_need_no_note(monkeypatch, which):
    plan = binding.RopePlan(64)
    w, s = Watch(monkeypatch), FakeStream()
    monkeypatch.setattr(binding, "RopePlan", lambda D: plan)
    s.cuda_stream = 5                                  # the current stream's handle
    call, shapes = results(w)[which]
    for stream in (None, s):
        w.made.clear()
        call(stream)
        assert [(x[0], x[2]) for x in w.made] == [(shape, None) for shape in shapes] and w.noted == []


def attention_case():
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = binding.KvCache(1, 600, 2, 64, 128, 4, 150)
    cache.k.normal_(generator=g), cache.v.normal_(generator=g)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    assert bool(binding.kv_reserve(cache, slots, 9000).all())
    binding.kv_commit(cache, slots, torch.tensor([8000, 5000, 100, 7001], dtype=torch.int32, device="cuda"), 9000)
    q = torch.randn(4, 8, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    return cache, slots, q


def take_what_was_dropped(sizes):
    """Blocks of these sizes from the current stream's pool, filled with NaN at once."""
    return [torch.full((n // 4,), float("nan"), device="cuda") for n in sizes for _ in range(3)]


@pytest.mark.gpu
def test_the_attention_on_a_stream_that_is_behind():
    cache, slots, q = attention_case()
    want = binding.tree_attn(cache, 0, slots, q)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    size, s = binding.tree_attn_workspace(cache, 4, 8, 16), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)             # some 10 ms
        binding.tree_attn(cache, 0, slots, q, out=out, stream=s)
        taken = take_what_was_dropped([size])
        s.synchronize()
        assert torch.equal(out, want)
        assert all(bool(x.isnan().all()) for x in taken)
    assert binding.kv_read_status(cache) == 0


@pytest.mark.gpu
def test_results_on_a_stream_that_is_behind():
    """The current stream is held up with a write to a block that is then dropped: a result may not be
    taken from it.  And a result that the current stream still has to read is not handed out again by its own
    stream, however soon it is dropped."""
    cache, slots, q = attention_case()
    plan, pos = binding.RopePlan(128), torch.arange(32, dtype=torch.int32, device="cuda")
    x = q.view(32, 16, 128)
    want = binding.rope(plan, pos, x)
    want_attn = binding.tree_attn(cache, 0, slots, q)
    work = torch.empty(binding.tree_attn_workspace(cache, 4, 8, 16), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)
        late = [torch.full_like(q, float("nan")) for _ in range(4)]
        del late                                       # free for the current stream, written in 10 ms
        got = binding.rope(plan, pos, x, stream=s)
        got_attn = binding.tree_attn(cache, 0, slots, q, workspace=work, stream=s)
        s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_attn, want_attn)
        torch.cuda._sleep(20_000_000)
        copy = torch.empty_like(got)
        copy.copy_(got)                                # reads `got` in 10 ms
        del got, got_attn
        for _ in range(4):
            binding.rope(plan, pos, -x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
    assert binding.kv_read_status(cache) == 0
