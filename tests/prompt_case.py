"""Packed prompts over a cache with scattered pages, and the 64-bit definition of their attention, for
the tests.  Bounds as in test_gpu_tree_attn.py: one rounding of the result (2^-8 of it in bf16, 2^-24
in fp32), with bf16 that of every probability (2^-8 of sum p |v|), and 2e-5 of sum p |v| for fp32 sums
of scores and of terms; lse 2e-5 absolute.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from gated_delta_rule_spec_gb300 import binding
from tests import attn_ref as ref

HALF_ULP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
FP32_NOISE = 2e-5


def attention(q, k_pool, v_pool, table, slots, lens, starts, scale):
    """(out, lse, spread) of q [N, HQ, D], float64: token t of row b sees its slot's committed tokens and the
    row's tokens 0..t.  Tokens of padding rows: zeros and -inf; tokens of no row: NaN."""
    N, HQ, D = q.shape
    G = HQ // k_pool.shape[1]
    out, spread, lse = (np.full(s, np.nan) for s in ((N, HQ, D), (N, HQ, D), (N, HQ)))
    for b, s in enumerate(slots):
        a, e = int(starts[b]), int(starts[b + 1])
        out[a:e], spread[a:e], lse[a:e] = 0, 0, -math.inf
        if s < 0 or a == e:
            continue
        n = int(lens[s])
        far = np.arange(n + e - a)[None] > n + np.arange(e - a)[:, None]
        for h in range(HQ):
            k, v = (ref.gather(p, table[s], n + e - a, h // G) for p in (k_pool, v_pool))
            x = np.where(far, -math.inf, (q[a:e, h] @ k.T) * scale)
            m = x.max(1, keepdims=True)
            p = np.exp(x - m)
            total = p.sum(1, keepdims=True)
            lse[a:e, h] = (m + np.log(total))[:, 0]
            p /= total
            out[a:e, h] = p @ v
            spread[a:e, h] = p @ np.abs(v)
    return out, lse, spread


class Prompts:
    """Rows of `counts` new tokens behind `lens` committed ones, one layer of a cache whose unused rows are
    poisoned.  `tail`: tokens behind the last row that no row owns; `lead`: before the first."""

    def __init__(self, seed, io, HQ, HKV, D, P, counts, lens, slots=None, layers=1, layer=0, poison=True, scale=None,
                 lead=0, tail=0):
        r = self.rng = np.random.default_rng(seed)
        self.io, self.HQ, self.D, self.P, self.layer = io, HQ, D, P, layer
        self.counts, self.lens = np.asarray(counts, np.int32), np.asarray(lens, np.int32)
        B = len(self.counts)
        self.slots = np.asarray(range(B) if slots is None else slots, np.int32)
        self.starts = (lead + np.concatenate([[0], np.cumsum(self.counts)])).astype(np.int32)
        self.N = int(self.starts[-1]) + tail
        self.scale = D ** -0.5 if scale is None else scale
        new = np.zeros(len(self.lens), np.int64)
        for b, s in enumerate(self.slots):
            if 0 <= s < len(self.lens):
                new[s] = self.counts[b]
        need = -(-(self.lens + new) // P)
        self.num_pages, max_pages = int(need.sum()) + 2, int(need.max()) + 1
        self.table, order, at = np.full((len(self.lens), max_pages), -1, np.int32), r.permutation(self.num_pages), 0
        for s, c in enumerate(need):
            self.table[s, :c] = order[at:at + c]
            at += c
        self.n_pages = need.astype(np.int32)
        shape = (layers, self.num_pages, HKV, P, D)
        self.k, self.v = ref.draw(r, shape, io), ref.draw(r, shape, io)
        if poison:   # what no token owns may be anything
            live = np.zeros((self.num_pages, P), bool)
            for s in range(len(self.lens)):
                i = np.arange(int(self.lens[s] + new[s]))
                live[self.table[s, i // P], i % P] = True
            dead = torch.from_numpy(~live)[None, :, None, :, None].expand(shape)
            for x, bad in ((self.k, math.nan), (self.v, math.inf)):
                x.masked_fill_(dead, bad)
        self.q = ref.draw(r, (self.N, HQ, D), io)
        self.cache = None

    def upload(self):
        t = {"k": self.k.cuda(), "v": self.v.cuda(), "page_table": torch.from_numpy(self.table).cuda(),
             "n_pages": torch.from_numpy(self.n_pages).cuda(), "length": torch.from_numpy(self.lens).cuda()}
        L, NP, HKV, P, D = self.k.shape
        self.cache = binding.KvCache(L, NP, HKV, P, D, len(self.lens), self.table.shape[1], self.io, tensors=t)
        return self.cache

    def row(self, slot, i):
        """(page, offset) of token i of a slot."""
        return int(self.table[slot, i // self.P]), i % self.P

    def call(self, **kw):
        cache = self.cache or self.upload()
        out = torch.full((self.N, self.HQ, self.D), 7.0, dtype=ref.TORCH[self.io], device="cuda")
        lse = torch.full((self.N, self.HQ), 7.0, device="cuda")
        binding.prompt_attn(cache, self.layer, torch.from_numpy(self.slots).cuda(), torch.from_numpy(self.starts).cuda(),
                            self.q.cuda(), scale=self.scale, out=out, lse=lse, **kw)
        return out, lse

    def expect(self):
        f = lambda x: x.double().numpy()  # noqa: E731
        return attention(f(self.q), f(self.k[self.layer]), f(self.v[self.layer]), self.table, self.slots, self.lens,
                         self.starts, self.scale)

    def bound(self, want, spread):
        p_round = HALF_ULP["bf16"] if self.io == "bf16" else 0.0
        return HALF_ULP[self.io] * np.abs(want) + (p_round + FP32_NOISE) * spread * (1 + 2.0 ** -8)

    def check(self, **kw):
        out, lse = self.call(**kw)
        assert binding.kv_read_status(self.cache) == 0
        want, want_lse, spread = self.expect()
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        nobody = np.isnan(want_lse)
        assert (got[nobody] == 7).all() and (gl[nobody] == 7).all()      # left as they were
        got, want, spread = (np.where(nobody[..., None], 0, x) for x in (got, want, spread))
        assert np.isfinite(got).all()
        worst = np.max(np.abs(got - want) - self.bound(want, spread), initial=-1.0)
        assert worst <= 0, (worst, np.max(np.abs(got - want)), np.argwhere(np.abs(got - want) > self.bound(want, spread))[:8])
        gl, want_lse = (np.where(nobody, 0, x) for x in (gl, want_lse))
        assert np.array_equal(np.isneginf(gl), np.isneginf(want_lse))
        fin = np.isfinite(want_lse)
        assert np.max(np.abs(gl[fin] - want_lse[fin]), initial=0.0) <= 2e-5
        return out, lse
