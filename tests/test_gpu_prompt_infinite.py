"""Prompt attention where scores are minus infinity: what the definition gives there (bounds: prompt_case.py)."""
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
