"""Appends to a slot whose page table holds an entry that is not a page where the window goes: the tokens
that would lie in it write nothing and their q is zero, all others are served, and with the entry
mended the same call makes up for it."""
import os

import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests import attn_ref as ref

@pytest.mark.gpu
@pytest.mark.parametrize("io,HQ,HKV,D,rot,layout", [("bf16", 4, 2, 64, 64, "half"), ("fp32", 3, 1, 32, 16, "interleaved"),
                                                    ("bf16", 2, 2, 40, 20, "half")])
@pytest.mark.parametrize("T,P,col", [(20, 16, 1), (20, 16, 2), (2, 16, 1), (300, 16, 19), (700, 32, 0), (1500, 16, 57)])
def test_append_leaves_the_tokens_of_a_bad_page_alone(io, HQ, HKV, D, rot, layout, T, P, col):
    """The first page, one in the middle or the last one of the window is bad."""
    at = 15                                                         # where the window starts
    need = -(-(at + T) // P)
    assert col < need
    cache = binding.KvCache(1, 3 * need + 1, HKV, P, D, 3, need, io)
    cache.k.zero_(), cache.v.zero_()
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    assert bool(binding.kv_reserve(cache, slots, at + T).all())
    binding.kv_commit(cache, slots, torch.full((3,), at, dtype=torch.int32, device="cuda"), at)
    qkv = torch.ones(3, T, HQ + 2 * HKV, D, dtype=ref.TORCH[io], device="cuda")
    part = qkv.split([HQ, HKV, HKV], 2)
    plan = binding.RopePlan(D, rot, layout=layout)
    good = binding.rope_append(plan, cache, 0, slots, *part)
    assert binding.kv_read_status(cache) == 0 and bool((good != 0).any(-1).all())
    k, v, page = cache.k.clone(), cache.v.clone(), int(cache.page_table[1, col])
    first, last = max(0, col * P - at), min(T, (col + 1) * P - at)  # the tokens of that page
    for bad in (-1, 3 * need + 1, 2147483647, -2147483648):
        cache.k.zero_(), cache.v.zero_()
        cache.page_table[1, col] = bad
        out = binding.rope_append(plan, cache, 0, slots, *part)
        assert binding.kv_read_status(cache) == binding.ST_PAGE_OOR
        q1, k1, v1 = good.clone(), k.clone(), v.clone()
        q1[1, first:last], k1[:, page], v1[:, page] = 0, 0, 0
        assert torch.equal(out, q1) and torch.equal(cache.k, k1) and torch.equal(cache.v, v1)
        if first > 0:                                               # a window that ends before the page
            counts = torch.tensor([T, first, T], dtype=torch.int32, device="cuda")
            out = binding.rope_append(plan, cache, 0, slots, *part, n_tokens=counts)
            assert binding.kv_read_status(cache) == 0
            assert torch.equal(out[1, :first], good[1, :first]) and bool((out[1, first:] == 0).all())
        cache.page_table[1, col] = page
        out = binding.rope_append(plan, cache, 0, slots, *part)
        assert binding.kv_read_status(cache) == 0
        assert torch.equal(out, good) and torch.equal(cache.k, k) and torch.equal(cache.v, v)


@pytest.mark.gpu
def test_append_one_token_of_many_rows():
    """Sixteen rows a block: each row's page is its own affair."""
    B = 5000
    cache = binding.KvCache(1, B, 1, 16, 16, B, 1, "bf16")
    cache.k.zero_(), cache.v.zero_()
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    assert bool(binding.kv_reserve(cache, slots, 1).all())
    r = np.random.default_rng(0)
    bad = torch.from_numpy(r.random(B) < 0.2).cuda()
    cache.page_table[bad] = B
    qkv = torch.ones(B, 1, 3, 16, dtype=torch.bfloat16, device="cuda")
    out = binding.rope_append(binding.RopePlan(16), cache, 0, slots, *qkv.split(1, 2))
    assert binding.kv_read_status(cache) == binding.ST_PAGE_OOR
    assert torch.equal((out != 0).any(-1)[:, 0, 0], ~bad)
    assert torch.equal((cache.v[0, :, 0, 0] != 0).any(-1), ~bad)


def test_the_header_says_so():
    text = " ".join(open(os.path.join(os.path.dirname(__file__), "..", "include", "gdn_spec.h")).read().replace(" * ", " ").split())
    entry = text[text.index("gdn_spec_rope_append -- a window's"):text.index("int gdn_spec_rope_append(")]
    assert "PAGE_OOR: the tokens whose place in the page table is no page write zeros to q_out only" in entry
