"""Values that are not finite in many of a block's pieces, one behind another: what a piece notes of them is its own."""
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests.prompt_case import Prompts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,HKV", [(128, 8), (64, 8), (256, 8)])
def test_a_later_tile_opens_a_note_that_an_earlier_piece_used(D, HKV):
    """160 rows of 128 tokens behind 64, 8 kv heads: some eight pieces a block, a head each, which use four notes in
    turn.  The values of token 100, in the tile that only the second half of the tokens sees, are infinite in every head, so
    every piece opens its note there; those of token 3, in the tile before, only in the first four heads.  So in the other
    heads the tokens up to 99 are as they were, bit for bit: nothing that an earlier piece noted reaches them."""
    B, n, committed = 160, 128, 64
    c = Prompts(61, "bf16", 2 * HKV, HKV, D, 64, counts=[n] * B, lens=[committed] * B, poison=False)
    want, wl = c.call()
    for t, heads in ((100, HKV), (3, HKV // 2)):
        pages, off = torch.from_numpy(c.table[:, (committed + t) // 64].astype(np.int64)).cuda(), (committed + t) % 64
        c.cache.v[0, pages, :heads, off, 5] = math.inf
    want, wl = want.view(B, n, HKV, 2, D), wl.view(B, n, HKV, 2)
    seen = torch.zeros(n, HKV, dtype=torch.bool, device="cuda")   # tokens that see an infinite value of a head
    seen[100:] = True
    seen[3:, :HKV // 2] = True
    for _ in range(10):
        out, lse = (x.view(y.shape) for x, y in zip(c.call(), (want, wl)))
        assert binding.kv_read_status(c.cache) == 0
        assert torch.equal(lse, wl)
        free = ~seen[None, :, :, None].expand(B, n, HKV, 2)
        assert torch.equal(out[free], want[free])
        assert torch.isposinf(out[~free][:, 5]).all()
        rest = torch.arange(D, device="cuda") != 5
        # The other dims of a removed row are added with a weight formed anew, one step of bf16 (2^-7 of it) off at most; the
        # weights sum to one, and both results are rounded (2^-8 of them each).
        a, b = out[~free][:, rest].float(), want[~free][:, rest].float()
        assert torch.isfinite(a).all()
        assert ((a - b).abs() <= 2.0 ** -7 * (b.abs() + float(c.v.abs().max()))).all()


@pytest.mark.parametrize("D", [128, 256])
def test_a_call_that_gives_up_beside_notes(D):
    """The wait limit at zero where every piece has values that are not finite: TIMEOUT, and the next call is right."""
    c = Prompts(62, "bf16", 8, 4, D, 64, counts=[128] * 40, lens=[64] * 40, poison=False)
    cache = c.upload()
    cache.v[:, :, :, 40, 1] = math.inf
    binding.set_wait_limit(0)
    try:
        c.call()
        st = binding.kv_read_status(cache)
    finally:
        binding.set_wait_limit(binding.WAIT_LIMIT_DEFAULT)
    assert st == binding.ST_TIMEOUT
    cache.v.copy_(c.v)
    c.check()
