"""Prompt attention where scores are minus infinity and where a weight vanishes beside an infinite value: what the definition
gives there (bounds: prompt_case.py)."""
import math

import numpy as np
import pytest
import torch

from tests.prompt_case import Prompts

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 4, 2, 128, 64), ("bf16", 2, 1, 64, 16), ("bf16", 4, 1, 256, 32), ("bf16", 6, 2, 96, 128), ("fp32", 4, 2, 128, 32),
          ("fp32", 2, 1, 256, 16)]


@pytest.mark.parametrize("io,HQ,HKV,D,P", SHAPES)
def test_a_token_whose_scores_are_all_minus_infinity(io, HQ, HKV, D, P):
    """There the softmax has no value: NaN, with an lse of -inf (zeros are for padding and refused rows).  One finite score
    among them takes the whole weight.  Rows of one block, and single tokens whose keys go over many blocks."""
    lens, counts = [0, 0, 40, 9000, 9000], [1, 150, 30, 1, 1]
    c = Prompts(51, io, HQ, HKV, D, P, counts, lens, poison=False)
    c.q[..., 0] = 1.0
    alone = {0: 0, 1: 100, 2: 69, 3: 9000, 4: None}      # the token of each slot whose key stays finite; slot 4: none
    for s, keep in alone.items():
        for i in range(lens[s] + counts[s]):
            if i != keep:
                page, off = c.row(s, i)
                c.k[0, page, :, off, 0] = -math.inf
    out, lse = c.call()
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    q, k, v = (x.double().numpy() for x in (c.q, c.k[0], c.v[0]))
    for s, keep in alone.items():
        for t in range(counts[s]):
            n = c.starts[s] + t
            if keep is None or lens[s] + t < keep:
                assert np.isnan(got[n]).all() and np.isneginf(gl[n]).all(), (s, t)
                continue
            page, off = c.row(s, keep)
            for h in range(HQ):
                g = h // (HQ // HKV)
                want, score = v[page, g, off], float(q[n, h] @ k[page, g, off]) * c.scale
                assert (np.abs(got[n, h] - want) <= c.bound(want, np.abs(want))).all(), (s, t, h)
                assert abs(gl[n, h] - score) <= 2e-5, (s, t, h)


@pytest.mark.parametrize("io,HQ,HKV,D,P", SHAPES)
@pytest.mark.parametrize("at", [0, 3, 130, 200])
def test_an_infinite_value_beside_a_weight_that_vanishes(io, HQ, HKV, D, P, at):
    """A weight of e^-200 is zero in 32 bits, and times infinity it is not finite, in whichever tile the key lies: the tokens
    that see it are not finite in that dim, whether others of their block see it or not; the rest are as ever."""
    c, clean = (Prompts(52, io, HQ, HKV, D, P, counts=[260], lens=[0], poison=False, scale=1.0) for _ in range(2))
    for x in (c, clean):
        x.q.zero_()
        x.q[..., 0] = 1.0
        x.k[..., 0] = 0.0
        page, off = x.row(0, at)
        if at:
            x.k[0, page, :, off, 0] = -200.0
        else:                                             # the first token sees nothing else: its weight is one
            x.k[..., 0] = 200.0
            x.k[0, page, :, off, 0] = 0.0
    c.v[0, page, :, off, 1] = math.inf
    got, want = c.call()[0].float().cpu().numpy(), clean.call()[0].float().cpu().numpy()
    assert np.array_equal(got[:at], want[:at]) and np.isfinite(want).all()
    assert not np.isfinite(got[at:, :, 1]).any()
    assert np.array_equal(np.delete(got, 1, 2), np.delete(want, 1, 2))
