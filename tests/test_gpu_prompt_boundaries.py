"""Prompt attention where its work is cut: chunks of prompts and windows behind one another on one cache, and contexts that are
gone through in several waves, against the 64-bit definition (torch, on the GPU, for its size).

Bounds as in prompt_case.py, of each output for itself: its rounding (2^-8 of it), that of the probabilities (2^-8 of
sum p |v|), 2e-5 of sum p |v| for the fp32 sums.  Values beside a cut are eight times as large as others, so that one
that is lost or counted twice is far outside: a test plants that in the definition."""
import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests.prompt_case import Prompts

pytestmark = pytest.mark.gpu


def definition(q, k, v, first, scale, without=None):
    """(out, bound) in 64 bits of q [n, HQ, D], the tokens first .. first + n of k, v [HKV, tokens, D]; without: a token that is
    left out where it is not the asking one."""
    n, HQ, _ = q.shape
    out, spread = (torch.empty(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    G, j, t = HQ // k.shape[0], torch.arange(k.shape[1], device="cuda"), first + torch.arange(n, device="cuda")[:, None]
    far = j > t
    if without is not None:
        far = far | ((j == without) & (j != t))
    for h in range(HQ):
        x = (q[:, h].double() @ k[h // G].double().T * scale).masked_fill(far, -np.inf)
        p = torch.exp(x - x.max(1, keepdim=True).values)
        p /= p.sum(1, keepdim=True)
        out[:, h], spread[:, h] = p @ v[h // G].double(), p @ v[h // G].double().abs()
    return out, 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2e-5) * spread * (1 + 2.0 ** -8)


def tokens_of(cache, slot, n):
    """Keys and values [HKV, n, D] of a slot's first n tokens."""
    page = cache.page_table[slot].long()
    i = torch.arange(n, device="cuda")
    return (x[0, page[i // cache.P], :, i % cache.P].transpose(0, 1) for x in (cache.k, cache.v))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    """One layer's normed append and attention, on a cache of its own."""

    def __init__(self, HQ, HKV, D, P):
        self.cache = binding.KvCache(1, 200, HKV, P, D, 4, 40)
        self.HQ, self.HKV, self.D = HQ, HKV, D
        self.plan = binding.RopePlan(D, D // 2, base=1.0e5)
        gen = torch.Generator(device="cuda").manual_seed(1)
        self.norms = [binding.HeadNorm(0.1 * torch.randn(D, generator=gen, device="cuda"), offset=1.0) for _ in range(2)]

    def append(self, slots, rows):
        counts = [len(r) for r in rows]
        starts, s = i32([sum(counts[:b]) for b in range(len(rows) + 1)]), i32(slots)
        assert bool(binding.kv_reserve(self.cache, s, max(counts), i32(counts)).all())
        q, k, v = torch.cat(rows).split([self.HQ, self.HKV, self.HKV], dim=1)
        return counts, starts, s, binding.norm_rope_append(self.plan, self.cache, 0, s, starts, q, k, v, *self.norms)

    def commit(self, slots, counts):
        binding.kv_commit(self.cache, slots, i32(counts), max(counts))
        assert binding.kv_read_status(self.cache) == 0

    def prompt(self, slots, rows):
        """rows: a list of [n, HQ + 2 HKV, D]; what the attention asked and gave, row by row."""
        counts, starts, s, q = self.append(slots, rows)
        out = binding.prompt_attn(self.cache, 0, s, starts, q)
        self.commit(s, counts)
        return list(zip(q.split(counts), out.split(counts)))

    def window(self, slots, rows):
        """The same of rows of T tokens each, through the tree attention."""
        counts, _, s, q = self.append(slots, rows)
        q = q.view(len(rows), counts[0], self.HQ, self.D)
        out = binding.tree_attn(self.cache, 0, s, q)
        self.commit(s, counts)
        return list(zip(q, out))


LENGTHS, CHUNK = [300, 1, 64, 129], 70


@pytest.mark.parametrize("HQ,HKV,D,P", [(8, 2, 64, 16), (8, 2, 128, 64), (4, 1, 256, 32), (6, 2, 96, 128)])
def test_chunks_and_windows_lose_no_token_and_count_none_twice(HQ, HKV, D, P):
    gen = torch.Generator(device="cuda").manual_seed(2)
    rows = [torch.randn(n, HQ + 2 * HKV, D, generator=gen, device="cuda").to(torch.bfloat16) for n in LENGTHS]
    edges = [[t for cut in range(0, n + 1, CHUNK) for t in (cut - 1, cut) if 0 <= t < n] for n in LENGTHS]
    for r, at in zip(rows, edges):
        r[at, HQ + HKV:] *= 8
    whole, chunks, trees = (Layer(HQ, HKV, D, P) for _ in range(3))
    asked, given = zip(*whole.prompt([0, 1, 2, 3], rows))
    pieces, order = [[] for _ in rows], [2, 0, 3, 1]
    for at in range(0, max(LENGTHS), CHUNK):               # some rows are done before others
        for b, x in zip(order, chunks.prompt(order, [rows[b][at:at + CHUNK] for b in order])):
            pieces[b].append(x)
    windows = [trees.window([0], [rows[0][at:at + 50]])[0] for at in range(0, 300, 50)]
    got = {"whole": given, "chunks": [torch.cat([o for _, o in p]) for p in pieces], "windows": [torch.cat([o for _, o in windows])]}
    assert torch.equal(torch.cat([q for q, _ in windows]), asked[0])
    for b, n in enumerate(LENGTHS):
        k, v = tokens_of(whole.cache, b, n)
        k2, v2 = tokens_of(chunks.cache, b, n)
        assert torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(torch.cat([q for q, _ in pieces[b]]), asked[b])
        want, bound = definition(asked[b], k, v, 0, D ** -0.5)
        for name, outs in got.items():
            if b < len(outs):
                assert ((outs[b].double() - want).abs() <= bound).all(), (name, b)
        for t in edges[b]:                                  # a definition that loses a token beside a cut is outside
            if t < n - 1:
                other, wide = definition(asked[b], k, v, 0, D ** -0.5, without=t)
                assert ((given[b].double() - other).abs() > wide).any(), (b, t)


@pytest.mark.parametrize("HQ,HKV,D,P,counts,lens", [(8, 8, 256, 64, [500, 1, 490], [13000, 5000, 12000]),
                                                    (6, 2, 256, 64, [300, 1, 250], [40000, 5000, 37000]),
                                                    (24, 8, 64, 64, [300, 1, 250], [33000, 7000, 40000]),
                                                    (16, 8, 128, 32, [400, 1, 380], [14000, 300, 20000])])
def test_several_waves(HQ, HKV, D, P, counts, lens):
    """Rows of more than two blocks of tokens whose keys and values are more than are gone through at a time (96 MB), beside a
    decoding row.  That the call plans several waves is seen from the workspace: one wave's is refused."""
    block = (128 if D == 256 else 256) // (HQ // HKV)       # tokens of a block at most
    full = [b for b, n in enumerate(counts) if n > 2 * block]
    assert len(full) == 2 and sum(counts) >= 2 * block * len(counts)
    assert sum(counts[b] + lens[b] for b in full) * HKV * D * 4 > 96 << 20
    c = Prompts(21, "bf16", HQ, HKV, D, P, counts=counts, lens=lens, poison=False)
    cache = c.upload()
    one = binding.prompt_attn_workspace(cache, 3, 1, HQ)
    with pytest.raises(binding.GdnSpecError):
        c.call(workspace=torch.empty(one, dtype=torch.uint8, device="cuda"))
    out, _ = c.call()
    assert binding.kv_read_status(cache) == 0
    for b, n in enumerate(counts):
        k, v = tokens_of(cache, b, lens[b] + n)
        at = slice(int(c.starts[b]), int(c.starts[b + 1]))
        want, bound = definition(c.q[at].cuda(), k, v, lens[b], c.scale)
        assert ((out[at].double() - want).abs() <= bound).all(), b
