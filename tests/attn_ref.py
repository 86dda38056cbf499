"""Plain 64-bit definitions of the softmax-attention layers' operators, for the tests: a
cache kept as Python lists and numpy arrays, attention row by row, rotary angles in
double precision.  Nothing here uses the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def draw(rng, shape, io):
    """Normal values as stored: a CPU tensor of the I/O type."""
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(TORCH[io])


def ancestors(parent) -> np.ndarray:
    """Masks of a tree whose node j hangs below parent[j] (-1: a root), as uint64."""
    m = np.zeros(len(parent), np.uint64)
    for j, p in enumerate(parent):
        m[j] = np.uint64(1 << j) | (m[p] if p >= 0 else np.uint64(0))
    return m


def random_tree(rng, T, reach=6):
    return [int(rng.integers(max(-1, j - reach), j)) for j in range(T)]


def pages_for(rng, lens, extra, P, num_pages, max_pages):
    """A page table that gives slot s room for lens[s] + extra tokens, pages in random order."""
    order, at = rng.permutation(num_pages), 0
    table = np.full((len(lens), max_pages), -1, np.int32)
    count = np.zeros(len(lens), np.int32)
    for s, n in enumerate(lens):
        c = -(-(int(n) + extra) // P)
        table[s, :c] = order[at:at + c]
        count[s] = c
        at += c
    return table, count


def gather(pool, table_row, n, h):
    """Rows 0..n-1 of a slot's head h: pool [num_pages, HKV, P, D] in 64 bits."""
    P = pool.shape[2]
    idx = np.arange(n)
    return pool[table_row[idx // P], h, idx % P]


def attention(q, k_pool, v_pool, table, slots, lens, masks, counts, scale):
    """(out, lse, spread): out [B, T, HQ, D], lse [B, T, HQ], spread = sum p |v|, which scales
    the error of rounded probabilities.  All float64; masks [B][T] python ints."""
    B, T, HQ, D = q.shape
    G = HQ // k_pool.shape[1]
    out, spread = np.zeros((B, T, HQ, D)), np.zeros((B, T, HQ, D))
    lse = np.full((B, T, HQ), -math.inf)
    for b in range(B):
        s = int(slots[b])
        if s < 0:
            continue
        n, c = int(lens[s]), int(counts[b])
        for h in range(HQ):
            k, v = (gather(p, table[s], n + c, h // G) for p in (k_pool, v_pool))
            for t in range(c):
                bits = int(masks[b][t])
                seen = np.array([True] * n + [bool(bits >> j & 1) for j in range(c)], bool)
                if not seen.any():
                    continue
                x = (k[seen] @ q[b, t, h]) * scale
                m = x.max()
                p = np.exp(x - m)
                lse[b, t, h] = m + math.log(p.sum())
                p = p / p.sum()
                out[b, t, h] = p @ v[seen]
                spread[b, t, h] = p @ np.abs(v[seen])
    return out, lse, spread


def frequencies(rot, base=1.0e4, scaling="none", factor=1.0, original=0.0, fast=32.0, slow=1.0, low=1.0,
                high=4.0):
    """(radians per position of each pair, factor on cos and sin)."""
    pairs = range(rot // 2)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in pairs]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "yarn":
        def pair_of(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair_of(fast)), 0)
        hi = min(math.ceil(pair_of(slow)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in pairs]
        return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1
    if scaling == "bands":
        mix = [min(max((original * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
        return [(1 - m) * x / factor + m * x for x, m in zip(f, mix)], 1.0
    return f, 1.0


def rotate(x, pos, freqs, mscale, rot, layout, transpose=False):
    """x [.., heads, D] in 64 bits, pos [..]: every head turned."""
    a = pos[..., None, None].astype(np.float64) * np.asarray(freqs)
    c, s = np.cos(a) * mscale, np.sin(a) * mscale
    if transpose:
        s = -s
    i = np.arange(rot // 2)
    i0, i1 = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y = np.array(x, np.float64)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i0] * s + x[..., i1] * c
    return y


class Pages:
    """The bookkeeping of the paged cache, one row after another: a page is free when its
    count of holders is zero, and the free page of lowest number is taken."""

    def __init__(self, num_pages, P, num_slots, max_pages):
        self.P, self.max_pages = P, max_pages
        self.ref = [0] * num_pages
        self.pages = [[] for _ in range(num_slots)]
        self.length = [0] * num_slots

    def _take(self, n):
        free = [p for p, r in enumerate(self.ref) if r == 0][:n]
        for p in free:
            self.ref[p] = 1
        return free

    def _serve(self, wants):
        """wants: (need or None) per row -> pages per row (None: refused)."""
        have, asked, got = sum(r == 0 for r in self.ref), 0, []
        for need in wants:
            if need is None:
                got.append(None)
                continue
            asked += need
            got.append(self._take(need) if need == 0 or asked <= have else None)
        return got

    def reserve(self, slots, T, counts=None):
        wants = []
        for b, s in enumerate(slots):
            n = T if counts is None else counts[b]
            if s < 0 or s >= len(self.pages) or not 0 <= n <= T:
                wants.append(None)
                continue
            need = -(-(self.length[s] + n) // self.P)
            wants.append(None if need > self.max_pages else max(0, need - len(self.pages[s])))
        got = self._serve(wants)
        for s, pages in zip(slots, got):
            if pages:
                self.pages[s] += pages
        return [int(g is not None) for g in got]

    def fork(self, src, dst):
        """Returns (done, copies): copies are (from page, to page, rows)."""
        wants = []
        for a, d in zip(src, dst):
            bad = a < 0 or d < 0 or a >= len(self.pages) or d >= len(self.pages)
            if bad or self.pages[d] or self.length[d]:
                wants.append(None)
            else:
                wants.append(1 if self.length[a] % self.P else 0)
        got, copies = self._serve(wants), []
        for a, d, pages in zip(src, dst, got):
            if pages is None:
                continue
            full = self.length[a] // self.P
            shared = self.pages[a][:full]
            for p in shared:
                self.ref[p] += 1
            if pages:
                copies.append((self.pages[a][full], pages[0], self.length[a] % self.P))
            self.pages[d] = shared + pages
            self.length[d] = self.length[a]
        return [int(g is not None) for g in got], copies

    def free(self, slots):
        for s in slots:
            if s < 0 or s >= len(self.pages):
                continue
            for p in self.pages[s]:
                self.ref[p] -= 1
            self.pages[s], self.length[s] = [], 0

    def moves(self, s, path):
        """(from, to) as (page, row) of the accepted drafts of slot s, in order."""
        n, P, pg = self.length[s], self.P, self.pages[s]
        return [((pg[(n + j) // P], (n + j) % P), (pg[(n + i) // P], (n + i) % P)) for i, j in enumerate(path)]

    def table(self):
        t = np.full((len(self.pages), self.max_pages), -1, np.int32)
        for s, pages in enumerate(self.pages):
            t[s, :len(pages)] = pages
        return t

    def bits(self):
        w = np.zeros((len(self.ref) + 31) // 32, np.uint32)
        for p, r in enumerate(self.ref):
            if r == 0:
                w[p // 32] |= np.uint32(1 << p % 32)
        return w.view(np.int32)
