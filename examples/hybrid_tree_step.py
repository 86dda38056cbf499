"""The speculative step of a hybrid model's two kinds of layers through the library.

Two softmax-attention layers over the paged cache, one feeding the other: three prompts go
into the cache in windows, each is forked, and then the same tokens are run twice, as one
drafted tree (rotary positions and append, tree attention, commit of the accepted path),
and one after another on the forks (windows of one token).

Beside them, one gated-delta-rule layer: it takes chains only, so no tree can go through it, and
it is shown by itself, with a chain of its own inputs, as long as the accepted path, through
verify, commit and fold.  Printed: how far the tree's outputs
on the accepted path are from the sequential ones, and the pages in use.

    python examples/hybrid_tree_step.py        (needs a GPU)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_delta_rule_spec_gb300 import binding  # noqa: E402


class AttentionLayer:
    """One softmax-attention layer: projections, rotary positions, the cache, the output."""

    def __init__(self, index, dim, HQ, HKV, D, plan, gen):
        self.index, self.HQ, self.HKV, self.D, self.plan = index, HQ, HKV, D, plan
        w = lambda *s: (torch.randn(*s, generator=gen, device="cuda") * s[0] ** -0.5).to(torch.bfloat16)  # noqa: E731
        self.qkv, self.out = w(dim, (HQ + 2 * HKV) * D), w(HQ * D, dim)

    def __call__(self, cache, slots, x, pos=None, mask=None, counts=None):
        B, T, _ = x.shape
        y = (x @ self.qkv).view(B, T, self.HQ + 2 * self.HKV, self.D)
        q, k, v = y.split([self.HQ, self.HKV, self.HKV], dim=2)
        q = binding.rope_append(self.plan, cache, self.index, slots, q, k, v, pos=pos, n_tokens=counts)
        o = binding.tree_attn(cache, self.index, slots, q, mask, counts)
        return x + o.view(B, T, -1) @ self.out


def tree(parent):
    """(ancestor masks as int64 words, depths) of a tree given by parents (-1: the last committed token)."""
    mask, depth = [], []
    for j, p in enumerate(parent):
        mask.append((1 << j) | (mask[p] if p >= 0 else 0))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return mask, depth


def delta_layer_step(chain, B, gen):
    """A window of random inputs through one gated-delta-rule layer, `chain` tokens of it accepted: verify,
    commit, fold."""
    H, HV, K, V, T = 4, 8, 128, 128, 4
    layer, cur = binding.SpecLayer(H, HV, K, V, T, 64, B), binding.SpecCursors(B)
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    A_log, dt = torch.zeros(HV, device="cuda"), torch.zeros(HV, device="cuda")
    out = binding.verify(layer, cur, slots, r(B, T, H, K), r(B, T, H, K), r(B, T, HV, V), r(B, T, HV), r(B, T, HV), A_log,
                         dt)
    binding.commit(cur, T, 64, slots, torch.full((B,), chain, dtype=torch.int32, device="cuda"))
    binding.fold(layer, cur, slots)
    assert binding.read_status(cur) == 0
    return out


def main(dim=256, HQ=8, HKV=2, D=64, P=16, prompts=(70, 5, 33), seed=0) -> float:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B = len(prompts)
    plan = binding.RopePlan(D, D // 2, scaling="yarn", base=1.0e4, factor=4.0, original=4096.0)
    layers = [AttentionLayer(i, dim, HQ, HKV, D, plan, gen) for i in range(2)]
    cache = binding.KvCache(len(layers), 64, HKV, P, D, num_slots=2 * B, max_pages=16)
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    forks = slots + B
    draw = lambda T: torch.randn(B, T, dim, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def forward(s, x, **kw):
        for layer in layers:
            x = layer(cache, s, x, **kw)
        return x

    # the prompts, in windows of at most 64 tokens of each
    for at in range(0, max(prompts), 64):
        counts = i32([max(0, min(64, n - at)) for n in prompts])
        assert bool(binding.kv_reserve(cache, slots, 64, counts).all())
        forward(slots, draw(64), counts=counts)
        binding.kv_commit(cache, slots, counts, 64)
    assert bool(binding.kv_fork(cache, slots, forks).all())

    # a tree of eight drafts; nodes 0, 2, 5, 7 are accepted
    parent, path = [-1, 0, 0, 1, 2, 2, 3, 5], [0, 2, 5, 7]
    mask, depth = tree(parent)
    T = len(parent)
    x = draw(T)
    assert bool(binding.kv_reserve(cache, slots, T).all())
    pos = cache.length[:B, None] + i32(depth)[None]
    y = forward(slots, x, pos=pos.contiguous(), mask=torch.tensor([mask] * B, device="cuda"))
    binding.kv_commit(cache, slots, i32([len(path)] * B), T, path=i32([path + [0] * (T - len(path))] * B))

    # the same tokens one after another on the forks
    worst = 0.0
    for node in path:
        assert bool(binding.kv_reserve(cache, forks, 1).all())
        z = forward(forks, x[:, node:node + 1].contiguous())
        binding.kv_commit(cache, forks, i32([1] * B), 1)
        worst = max(worst, float((z[:, 0].float() - y[:, node].float()).abs().max()))
    assert torch.equal(cache.length[:B], cache.length[B:]) and binding.kv_read_status(cache) == 0
    delta_layer_step(len(path), B, gen)
    used = int((cache.ref > 0).sum())
    binding.kv_free(cache, torch.cat([slots, forks]))
    assert int((cache.ref > 0).sum()) == 0 and binding.kv_read_status(cache) == 0
    moved = float((y.float() - x.float()).abs().max())
    assert moved > 0.1                                   # the layers did something
    print(f"tree against one after another: max-abs {worst:.2e} (the layers move the inputs by up to {moved:.1f}); "
          f"pages in use {used} of {cache.num_pages}")
    return worst


if __name__ == "__main__":
    main()
