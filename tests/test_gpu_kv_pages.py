"""The pages of the softmax-attention cache against the bookkeeping of tests/attn_ref.py:
tables, counts, holders, free bits and every key and value row, bit for bit, over
random sequences of reserve, fork, commit and free."""
import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Both:
    """The same cache on both sides."""

    def __init__(self, seed, layers, pages, HKV, P, D, slots, max_pages, io="bf16"):
        self.rng = np.random.default_rng(seed)
        self.cache = binding.KvCache(layers, pages, HKV, P, D, slots, max_pages, io)
        self.k, self.v = (ref.draw(self.rng, (layers, pages, HKV, P, D), io) for _ in range(2))
        self.cache.k.copy_(self.k), self.cache.v.copy_(self.v)
        self.ref = ref.Pages(pages, P, slots, max_pages)

    def check(self):
        c, r = self.cache, self.ref
        assert np.array_equal(c.page_table.cpu().numpy(), r.table())
        assert c.n_pages.tolist() == [len(p) for p in r.pages]
        assert c.length.tolist() == r.length
        assert c.ref.tolist() == r.ref
        assert np.array_equal(c.free_bits.cpu().numpy(), r.bits())
        assert torch.equal(c.k.cpu(), self.k) and torch.equal(c.v.cpu(), self.v)

    def reserve(self, slots, T, counts=None):
        done = binding.kv_reserve(self.cache, dev(slots), T, None if counts is None else dev(counts))
        assert done.tolist() == self.ref.reserve(list(slots), T, counts)

    def fork(self, src, dst):
        done = binding.kv_fork(self.cache, dev(src), dev(dst))
        want, copies = self.ref.fork(list(src), list(dst))
        assert done.tolist() == want
        for x in (self.k, self.v):
            for a, b, n in copies:
                x[:, b, :, :n] = x[:, a, :, :n]

    def commit(self, slots, T, paths):
        acc = [len(p) for p in paths]
        path = np.zeros((len(slots), T), np.int32)
        for i, p in enumerate(paths):
            path[i, :len(p)] = p
        binding.kv_commit(self.cache, dev(slots), dev(acc), T, path=dev(path))
        for s, p in zip(slots, paths):
            if s < 0:
                continue
            for (fp, fo), (tp, to) in self.ref.moves(s, p):
                for x in (self.k, self.v):
                    x[:, tp, :, to] = x[:, fp, :, fo].clone()
            self.ref.length[s] += len(p)

    def free(self, slots):
        binding.kv_free(self.cache, dev(slots))
        self.ref.free(list(slots))


@pytest.mark.parametrize("io,HKV,P,D,layers", [("bf16", 2, 16, 64, 3), ("fp32", 1, 32, 40, 2), ("bf16", 3, 128, 8, 1)])
@pytest.mark.parametrize("seed", range(3))
def test_random_lives(io, HKV, P, D, layers, seed):
    b = Both(seed, layers, 67, HKV, P, D, 13, 9, io)
    r, T = b.rng, 24
    for step in range(40):
        slots = [int(s) for s in r.permutation(13)[:int(r.integers(1, 9))]]
        kind = int(r.integers(0, 4))
        if kind == 0:
            if r.random() < 0.3:
                slots[0] = -1
            counts = [int(x) for x in r.integers(0, T + 1, len(slots))]
            b.reserve(slots, T, counts if r.random() < 0.5 else None)
        elif kind == 1:
            empty = [s for s in range(13) if not b.ref.pages[s]]
            full = [s for s in range(13) if b.ref.length[s]]
            if empty and full:
                dst = empty[:int(r.integers(1, len(empty) + 1))]
                b.fork([int(r.choice(full)) for _ in dst], dst)
        elif kind == 2:
            paths, at = [], []
            for s in slots:
                room = len(b.ref.pages[s]) * P - b.ref.length[s]
                n = min(T, room)
                m = int(r.integers(0, n + 1)) if n > 0 else 0
                paths.append(sorted(int(x) for x in r.permutation(n)[:m]))
                at.append(s)
            b.commit(at, T, paths)
        else:
            b.free(slots[:2])
        assert binding.kv_read_status(b.cache) in (0, binding.ST_NO_PAGES)
    b.check()


def test_refused_rows():
    b = Both(9, 1, 8, 1, 16, 8, 6, 4)
    c = b.cache
    b.reserve([0, 1], 48)                                  # six pages of eight
    b.check()
    # the third row asks for three pages of two: refused; so is the fourth, whatever it lacks behind it
    b.reserve([0, 1, 2, 3], 48)
    assert binding.kv_read_status(c) == binding.ST_NO_PAGES
    b.reserve([2], 65)                                     # five columns of four
    assert binding.kv_read_status(c) == binding.ST_NO_PAGES
    b.reserve([4, 17], 16, [16, 16])
    assert binding.kv_read_status(c) == binding.ST_SLOT_OOR
    b.reserve([5], 16, [17])
    assert binding.kv_read_status(c) == binding.ST_ACCEPT_RANGE
    b.check()
    b.commit([0], 40, [list(range(1, 21))])
    b.fork([0, 0], [1, 3])                                 # slot 1 holds pages: busy; one page is left for slot 3
    assert binding.kv_read_status(c) == binding.ST_SLOT_BUSY
    b.check()
    b.fork([0], [5])                                       # none left
    assert binding.kv_read_status(c) == binding.ST_NO_PAGES
    b.check()
    before = [t.clone() for t in (c.k, c.v, c.length)]
    T = 8
    bad = [([3, 2, 4], 3), ([0, 0, 1], 3), ([0, 1, 8], 3), ([-1, 0, 1], 3), ([0, 1, 2147483647], 3), ([0] * 8, 9),
           ([0] * 8, -1)]
    for p, n in bad:
        path = dev([(p + [0] * T)[:T]])
        binding.kv_commit(c, dev([0]), dev([n]), T, path=path)
        assert binding.kv_read_status(c) == binding.ST_ACCEPT_RANGE
    binding.kv_commit(c, dev([0]), dev([30]), 40, path=dev([list(range(9, 39)) + [0] * 10]))
    assert binding.kv_read_status(c) == binding.ST_NO_PAGES   # 20 + 39 rows in three pages
    binding.kv_commit(c, dev([0, 3]), dev([29, -2]), 40)
    assert binding.kv_read_status(c) == binding.ST_NO_PAGES | binding.ST_ACCEPT_RANGE
    assert all(torch.equal(x, y) for x, y in zip(before, (c.k, c.v, c.length)))


def test_corrupt_counts_are_reported():
    b = Both(10, 1, 8, 1, 16, 8, 4, 4)
    b.reserve([0, 1], 32)
    c = b.cache
    c.length[0] = 33
    for call in (lambda: binding.kv_reserve(c, dev([0]), 1), lambda: binding.kv_free(c, dev([0])),
                 lambda: binding.kv_fork(c, dev([0]), dev([3])), lambda: binding.kv_commit(c, dev([0]), dev([0]), 4)):
        call()
        assert binding.kv_read_status(c) == binding.ST_CURSOR_CORRUPT
    c.length[0] = 0
    c.page_table[1, 1] = 1000
    binding.kv_free(c, dev([1]))
    assert binding.kv_read_status(c) == binding.ST_PAGE_OOR
    c.page_table[0, 0] = 7                                  # a page that nobody holds
    binding.kv_free(c, dev([0]))
    assert binding.kv_read_status(c) == binding.ST_CURSOR_CORRUPT
    assert int(c.ref[7]) == 0


def test_many_pages_and_rows():
    """More words of free bits and more rows than one slice of the allocating block; every page is handed
    out, lowest first."""
    pages, slots, P = 70001, 3000, 16
    c = binding.KvCache(1, pages, 1, P, 8, slots, 40)
    s = torch.arange(slots, dtype=torch.int32, device="cuda")
    n = torch.from_numpy(np.random.default_rng(0).integers(0, 24 * P, slots).astype(np.int32)).cuda()
    done = binding.kv_reserve(c, s, 24 * P, n)
    assert bool(done.all()) and binding.kv_read_status(c) == 0
    need = (n.long() + P - 1) // P
    assert torch.equal(c.n_pages.long(), need)
    held = c.page_table[c.page_table >= 0]
    assert torch.equal(held, torch.arange(int(need.sum()), dtype=torch.int32, device="cuda"))
    binding.kv_free(c, s[::2].contiguous())
    assert int((c.ref == 0).sum()) == pages - int(need[1::2].sum())
    bits = sum(bin(x & 0xffffffff).count("1") for x in c.free_bits.tolist())
    assert bits == pages - int(need[1::2].sum())
    again = binding.kv_reserve(c, s[::2].contiguous(), 24 * P)
    want = torch.cumsum(torch.full((slots // 2,), 24), 0) <= bits
    assert torch.equal(again.cpu().bool(), want)
    binding.kv_init(c)
    assert int(c.n_pages.sum()) == 0 and int(c.ref.sum()) == 0 and bool((c.page_table == -1).all())
    assert sum(bin(x & 0xffffffff).count("1") for x in c.free_bits.tolist()) == pages


def test_stream_order_with_foreign_kernels():
    """Inputs written by the kernel just before each dependently launched call."""
    b = Both(12, 2, 64, 2, 16, 64, 8, 16)
    acc, path = dev([0] * 4), dev(np.zeros((4, 8)))
    slots = [0, 1, 2, 3]
    for step in range(12):
        b.reserve(slots, 8)
        paths = [sorted(int(x) for x in b.rng.permutation(8)[:int(b.rng.integers(1, 9))]) for _ in slots]
        full = np.zeros((4, 8), np.int32)
        for i, p in enumerate(paths):
            full[i, :len(p)] = p
        src_p, src_a = dev(full), dev([len(p) for p in paths])
        path.zero_(), acc.zero_()
        path.add_(src_p), acc.add_(src_a)
        binding.kv_commit(b.cache, dev(slots), acc, 8, path=path)
        for s, p in zip(slots, paths):
            for (fp, fo), (tp, to) in b.ref.moves(s, p):
                for x in (b.k, b.v):
                    x[:, tp, :, to] = x[:, fp, :, fo].clone()
            b.ref.length[s] += len(p)
        b.check()
    assert binding.kv_read_status(b.cache) == 0
