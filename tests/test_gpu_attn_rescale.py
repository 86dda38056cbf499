"""Attention whose running maximum climbs along the context, so that sums taken so far are rescaled.

A block walks many tiles of an item here, and in every item some query rows meet, at random
places, a key whose score stands 8.5 to 11 powers of two above all before it: the
tensor-core kernel then moves the row's maximum (it does so from 8 on) and scales what it has
summed.  About as much weight lies on the plain keys before and behind such a key as
on the key, so a sum that is scaled wrongly, or not at all, is off by a large part of itself.
Bounds as in test_gpu_tree_attn.py (scores stay below 16 here too); the 64-bit
definition runs on the GPU, the contexts being long.
"""
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests import attn_ref as ref
from tests.test_gpu_tree_attn import FP32_NOISE, HALF_ULP, Case

LOG2E = 1.0 / math.log(2.0)


def climbing(case, per_item=24):
    """Plain keys of small scores, and `per_item` keys in each (row, kv head) that lie along a query row."""
    r = np.random.default_rng(1234)
    T, G, D = case.T, case.HQ // case.k.shape[2], case.D
    case.k.mul_(0.5)
    for b, s in enumerate(case.slots):
        n = int(case.lens[s])
        for h in range(case.k.shape[2]):
            for at in r.choice(n, min(per_item, n), replace=False):
                t, g = int(r.integers(0, T)), int(r.integers(0, G))
                q = case.q[b, t, h * G + g].double()
                # scale log2(e) <q, k> = climb
                k = q * float(r.uniform(8.5, 11.0)) / (LOG2E * case.scale * float(q @ q))
                case.k[case.layer, int(case.table[s, at // case.P]), h, int(at % case.P)] = k.to(case.k.dtype)
    return case


def definition(case):
    """(out, lse, spread) in 64 bits, by torch on the device of the case's cache."""
    cache = case.cache
    B, T, HQ, D = case.q.shape
    HKV = cache.HKV
    G = HQ // HKV
    q = case.q.cuda().double()
    out, spread = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, T, HQ), -math.inf, dtype=torch.float64, device="cuda")
    for b, s in enumerate(case.slots):
        n, c = int(case.lens[s]), int(case.counts[b])
        i = torch.arange(n + c, device="cuda")
        page = cache.page_table[int(s)].long()[i // case.P]
        seen = torch.ones(c, n + c, dtype=torch.bool)
        seen[:, n:] = torch.tensor([[bool(case.masks[b][t] >> j & 1) for j in range(c)] for t in range(c)])
        seen = seen.cuda()
        for h in range(HKV):
            k, v = (x[case.layer][page, h, i % case.P].double() for x in (cache.k, cache.v))
            heads = slice(h * G, (h + 1) * G)
            x = torch.einsum("tgd,nd->tgn", q[b, :c, heads], k) * case.scale
            x = x.masked_fill(~seen[:, None], -math.inf)
            p = torch.softmax(x, -1)
            lse[b, :c, heads] = torch.logsumexp(x, -1)
            out[b, :c, heads] = p @ v
            spread[b, :c, heads] = p @ v.abs()
    return out, lse, spread


@pytest.mark.gpu
@pytest.mark.parametrize("io,T,HQ,HKV,D,P,rows,length", [
    ("bf16", 8, 4, 2, 64, 16, 6, 15000), ("bf16", 1, 8, 4, 64, 64, 3, 14000),          # 64 dims, one query tile
    ("bf16", 64, 8, 2, 64, 64, 5, 16000), ("bf16", 33, 8, 1, 64, 32, 9, 18000),        # two query tiles
    ("bf16", 8, 8, 2, 128, 64, 6, 15000), ("bf16", 1, 32, 8, 128, 128, 2, 12000),      # 128 dims
    ("bf16", 5, 6, 3, 96, 16, 4, 14000),
    ("bf16", 64, 8, 2, 128, 128, 5, 16000), ("bf16", 40, 16, 2, 128, 16, 4, 13000),
    ("bf16", 8, 16, 2, 256, 64, 6, 15000), ("bf16", 48, 8, 1, 256, 32, 8, 16000),      # 256 dims, one stream
    ("fp32", 8, 4, 2, 128, 64, 4, 9000), ("fp32", 16, 2, 1, 64, 16, 4, 9000)])
def test_the_maximum_climbs_along_the_context(io, T, HQ, HKV, D, P, rows, length):
    lens = [length - 977 * i for i in range(rows)]
    # a block's chunk is many tiles of 64 keys even if all 152 SMs take one
    assert sum(lens) * HKV / 64 / 152 >= (8 if io == "bf16" else 3)
    case = climbing(Case(31, io, T, HQ, HKV, D, P, lens))
    out, lse = case.call()
    assert binding.kv_read_status(case.cache) == 0
    want, want_lse, spread = definition(case)
    rounding = HALF_ULP["bf16"] if io == "bf16" else 0.0
    bound = HALF_ULP[io] * want.abs() + (rounding + FP32_NOISE) * spread * (1 + 2.0 ** -8)
    err = (out.double() - want).abs()
    assert bool(torch.isfinite(out).all())
    assert bool((err <= bound).all()), float((err - bound).max())
    assert float((lse.double() - want_lse).abs().max()) <= 2e-5


def walk(s, v, mistake=None, grow=8.0, tile=64):
    """One query row as a block walks it, in 64 bits: scores in powers of two, the maximum moved only when
    a tile's is more than `grow` above it.  Returns (output, how often sums were rescaled)."""
    m, l, o, moved = -math.inf, 0.0, np.zeros(v.shape[1]), 0
    for a in range(0, len(s), tile):
        x, top = s[a:a + tile], s[a:a + tile].max()
        if top > m + grow:
            al = 0.0 if m == -math.inf else 2.0 ** (m - top)
            if a > 0:
                moved += 1
                if mistake != "sums stay":
                    o = o * al
                if mistake == "sums lost":
                    o = o * 0
            l, m = l * al, top
        p = 2.0 ** (x - m)
        l, o = l + p.sum(), o + p @ v[a:a + tile]
    return o / l, moved


def test_the_keys_above_show_a_wrong_rescale():
    """On the CPU: rows that meet such a key rescale, and a definition that forgets or loses the sums is out of
    the bounds that the GPU test holds the kernels to."""
    case = climbing(Case(31, "bf16", 4, 4, 2, 64, 16, [2000, 1500], poison=False))
    found = {"sums stay": 0, "sums lost": 0}
    for b, s in enumerate(case.slots):
        n = int(case.lens[s])
        for h in range(case.HQ):
            k, v = (ref.gather(x[0].double().numpy(), case.table[s], n, h // 2) for x in (case.k, case.v))
            for t in range(case.T):
                x = k @ case.q[b, t, h].double().numpy() * case.scale * LOG2E
                p = 2.0 ** (x - x.max())
                want, spread = p @ v / p.sum(), p @ np.abs(v) / p.sum()
                got, moved = walk(x, v)
                assert np.allclose(got, want, rtol=0, atol=1e-12)
                bound = HALF_ULP["bf16"] * np.abs(want) + (HALF_ULP["bf16"] + FP32_NOISE) * spread * (1 + 2.0 ** -8)
                for mistake in found:
                    wrong, _ = walk(x, v, mistake)
                    if moved and (np.abs(wrong - want) > bound).any():
                        found[mistake] += 1
    assert min(found.values()) >= 12, found
