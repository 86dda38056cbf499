"""The sizes up to which the softmax-attention layers' calls go: the header names every limit, the call at
it is taken and the one past it refused (no rows, so nothing is launched)."""
import ctypes
import os
import re

import pytest

from gated_delta_rule_spec_gb300 import binding
from tests.test_attn_validation import EINVAL, EUNSUP, FAKE, OK, attn, cache, lib, plan  # noqa: F401

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "gdn_spec.h")


def entry(first, last):
    """The header's comment between two texts, without its line breaks."""
    text = re.sub(r"\s+", " ", re.sub(r"\n \* ?", " ", open(HEADER).read()))
    return text[text.index(first):text.index(last)]


def test_layers_and_heads(lib):
    assert "n_layers * HKV is at most 2^20" in entry("The cache of all softmax-attention layers", "gdn_spec_kv_cache;")
    for layers, heads, want in ((1 << 20, 1, OK), (1 << 10, 1 << 10, OK), ((1 << 20) + 1, 1, EUNSUP), (3, 349526, EUNSUP)):
        c = cache(n_layers=layers, HKV=heads)
        assert lib.gdn_spec_kv_free(ctypes.byref(c), FAKE, 0, None) == want


def test_heads_a_group(lib):
    assert "HQ / HKV is at most 4096" in entry("gdn_spec_tree_attn -- softmax", "int gdn_spec_tree_attn(")
    assert attn(lib, cache(), HQ=2 * 4096) == OK and attn(lib, cache(), HQ=2 * 4097) == EUNSUP


def test_rows_of_the_pool_on_the_tensor_cores(lib):
    assert "n_layers * num_pages * HKV * P below 2^31" in entry("Two kernels (gdn_spec_tree_attn_path)", "int gdn_spec_tree_attn(")
    for pages, want in (((1 << 31) // (2 * 64 * 4) - 1, b"tc"), ((1 << 31) // (2 * 64 * 4), b"generic")):
        c = cache(n_layers=4, HKV=2, P=64, num_pages=pages)
        assert lib.gdn_spec_tree_attn_path(ctypes.byref(c), 4, 8) == want


def test_rows_of_a_reserve(lib):
    assert "B * max_pages is below 2^31" in entry("gdn_spec_kv_reserve -- pages", "int gdn_spec_kv_reserve(")
    c = cache(P=16, max_pages=1 << 18)
    assert lib.gdn_spec_kv_reserve(ctypes.byref(c), FAKE, 8192, 4, None, FAKE, None) == EUNSUP


def test_elements_of_a_token(lib):
    assert "at least heads * D, which is at most 2^22" in entry("gdn_spec_rope -- out = R x", "int gdn_spec_rope(")
    assert "B * T is below 2^31 and (HQ + 2 HKV) * D at most 2^22" in entry("gdn_spec_rope_append -- a window", "int gdn_spec_rope_append(")
    p, s = plan(), 1 << 23

    def rope(heads):
        return lib.gdn_spec_rope(ctypes.byref(p), 0, heads, 0, FAKE, FAKE, s, FAKE + 65536, s, 0, None)

    def append(HQ, B=0, T=4):
        return lib.gdn_spec_rope_append(ctypes.byref(p), ctypes.byref(cache()), 0, FAKE, B, T, None, None, HQ, FAKE, s,
                                        FAKE, s, FAKE, s, FAKE, None)

    assert rope(1 << 15) == OK and rope((1 << 15) + 1) == EUNSUP
    assert append((1 << 15) - 4) == OK and append((1 << 15) - 3) == EUNSUP
    assert append(8, 1 << 25, 64) == EUNSUP


def test_scale(lib):
    """Scores are taken in powers of two: a scale whose product with log2(e) is no fp32 number gave NaN."""
    top = 3.4028234663852886e38 / 1.4426950408889634
    assert "scale > 0, and scale * log2(e) a finite fp32 number" in entry("gdn_spec_tree_attn -- softmax", "int gdn_spec_tree_attn(")
    for scale, want in ((0.999 * top, OK), (1.001 * top, EINVAL), (3.4e38, EINVAL), (1e-45, OK)):
        assert attn(lib, cache(), scale=scale) == want, scale


def test_factor_on_cos_and_sin(lib):
    """The plan keeps the factor in fp32, where it has to be finite."""
    assert plan(8, 2, freqs=[1.0], mscale=3e38).mscale > 0
    for mscale in (1e39, -1e39, 1e300):
        with pytest.raises(binding.GdnSpecError):
            plan(8, 2, freqs=[1.0], mscale=mscale)


def test_a_plans_dims_are_the_descriptors(lib):
    """rope() checks x against the plan's head dim, the kernel reads the descriptor's: one number."""
    p = binding.RopePlan(128, 64)
    assert (p.D, p.rot) == (p.desc().D, p.desc().rot) == (128, 64)
    with pytest.raises(AttributeError):
        p.D = 64
    with pytest.raises(AttributeError):
        p.rot = 32
    assert binding.RopePlan(64).rot == 64
