"""Prompts and the tokens behind them through two softmax-attention layers, as they are used: reserve, then per layer
the packed append and the attention, then commit.  The same tokens whole, in chunks, beside decoding rows, and as
windows through the tree attention give the same activations.

Activations are some 4 at most; each of the two layers rounds its projections, normed heads, probabilities, outputs and
residual to bf16 (2^-8 of the value each), which leaves a few times 2^-8 of 4."""
import os
import sys

import pytest
import torch

from gated_delta_rule_spec_gb300 import binding

pytestmark = pytest.mark.gpu

BOUND = 8 * 4 * 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import hybrid_tree_step
    finally:
        sys.path.pop(0)
    return hybrid_tree_step


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    def __init__(self, example, HQ, HKV, D, P, slots):
        gen = torch.Generator(device="cuda").manual_seed(1)
        plan = binding.RopePlan(D, D // 2, base=1.0e5)
        self.layers = [example.AttentionLayer(i, 256, HQ, HKV, D, plan, gen) for i in range(2)]
        self.cache = binding.KvCache(2, 400, HKV, P, D, slots, 40)

    def prompt(self, slots, x):
        """x: a list of [n, 256], n may be 0: the rows' activations."""
        counts = [len(r) for r in x]
        starts, s = i32([sum(counts[:b]) for b in range(len(counts) + 1)]), i32(slots)
        assert bool(binding.kv_reserve(self.cache, s, max(counts), i32(counts)).all())
        h = torch.cat(x)
        for layer in self.layers:
            h = layer.prompt(self.cache, s, starts, h)
        binding.kv_commit(self.cache, s, i32(counts), max(counts))
        assert binding.kv_read_status(self.cache) == 0
        return h.split(counts)

    def window(self, slots, x):
        """x [B, T, 256] as a chain through the tree attention."""
        s = i32(slots)
        assert bool(binding.kv_reserve(self.cache, s, x.shape[1]).all())
        for layer in self.layers:
            x = layer(self.cache, s, x)
        binding.kv_commit(self.cache, s, i32([x.shape[1]] * len(slots)), x.shape[1])
        assert binding.kv_read_status(self.cache) == 0
        return x


def far(a, b):
    return float((a.float() - b.float()).abs().max())


@pytest.mark.parametrize("HQ,HKV,D,P", [(8, 2, 64, 16), (8, 2, 128, 64), (4, 1, 256, 32), (6, 3, 96, 128)])
def test_whole_in_chunks_and_as_windows(example, HQ, HKV, D, P):
    gen = torch.Generator(device="cuda").manual_seed(2)
    lengths = [300, 1, 64, 129]
    x = [torch.randn(n, 256, generator=gen, device="cuda").to(torch.bfloat16) for n in lengths]
    whole = Model(example, HQ, HKV, D, P, 4)
    y = whole.prompt([0, 1, 2, 3], x)
    assert all(far(a, b) > 0.1 for a, b in zip(x, y))                       # the layers did something

    # in chunks of 70 tokens, rows in another order, some of them done before others
    chunks = Model(example, HQ, HKV, D, P, 4)
    got = [[] for _ in lengths]
    for at in range(0, 300, 70):
        order = [2, 0, 3, 1]
        for b, z in zip(order, chunks.prompt(order, [x[b][at:at + 70] for b in order])):
            got[b].append(z)
    for b in range(4):
        assert far(torch.cat(got[b]), y[b]) <= BOUND
    assert torch.equal(chunks.cache.length, whole.cache.length)

    # as windows of 50 drafted tokens through the tree attention
    trees = Model(example, HQ, HKV, D, P, 4)
    z = torch.cat([trees.window([0], x[0][None, at:at + 50]) for at in range(0, 300, 50)], 1)
    assert far(z[0], y[0]) <= BOUND

    # the next token of every row: through the packed call, beside a new prompt, and as windows of one
    step = torch.randn(4, 256, generator=gen, device="cuda").to(torch.bfloat16)
    packed = whole.prompt([3, 2, 1, 0], [step[b:b + 1] for b in (3, 2, 1, 0)])
    single = chunks.window([0, 1, 2, 3], step[:, None])
    for b in range(4):
        assert far(packed[3 - b], single[b]) <= BOUND


def test_a_step_captured_once_follows_the_counts(example):
    """A mixed step in a graph: the tensors' sizes are the graph's, the rows' counts, slots and lengths are read on the
    device at each replay."""
    m = Model(example, 8, 2, 128, 64, 4)
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda n: torch.randn(n, 256, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, starts, slots, counts = draw(200), i32([0, 0, 0, 0]), i32([0, 1, 2]), i32([0, 0, 0])
    layer, cache = m.layers[0], m.cache

    def step():
        done = binding.kv_reserve(cache, slots, 200, counts)
        y = layer.prompt(cache, slots, starts, x)
        binding.kv_commit(cache, slots, counts, 200)
        return y, done

    step()                                                                  # (kernels loaded before the capture)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, done = step()
    other = Model(example, 8, 2, 128, 64, 4)
    for rows in ([130, 0, 1], [1, 60, 90], [1, 1, 1], [0, 200, 0]):
        counts.copy_(i32(rows))
        starts.copy_(i32([sum(rows[:b]) for b in range(4)]))
        new = draw(200)
        x.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        assert bool(done.all()) and binding.kv_read_status(cache) == 0
        n = sum(rows)
        assert bool(binding.kv_reserve(other.cache, slots, 200, counts).all())
        want = other.layers[0].prompt(other.cache, slots, starts, new[:n])
        binding.kv_commit(other.cache, slots, counts, 200)
        assert torch.equal(y[:n], want)
    assert torch.equal(cache.length, other.cache.length)
