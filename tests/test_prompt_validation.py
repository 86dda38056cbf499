"""Host-side checks of the packed prompts' entry points, without a GPU: every call here fails validation or has nothing
to do, so the fake (aligned, never dereferenced) device pointers are never used.  And the limits that the header
names, at them and one past."""
import ctypes
import math
import os
import re

import pytest

from gated_delta_rule_spec_gb300 import binding
from tests.test_attn_limits import entry
from tests.test_attn_validation import BAD_CACHES, EALIGN, EDTYPE, EINVAL, EUNSUP, FAKE, MIS, OK, cache, lib, plan  # noqa: F401

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "gdn_spec.h")


def norm(weight=FAKE, eps=1e-6, offset=0.0):
    return binding.HeadNormDesc(weight, eps, offset)


def ref(x):
    return None if x is None else ctypes.byref(x)


def attn(lib, c, layer=0, slot=FAKE, starts=FAKE, B=1, N=0, HQ=8, q=FAKE, scale=0.1, out=FAKE, ws=FAKE, n=1 << 40):
    return lib.gdn_spec_prompt_attn(ref(c), layer, slot, starts, B, N, HQ, q, scale, out, None, ws, n, None)


def append(lib, c=None, p=None, qn=None, kn=None, layer=0, slot=FAKE, starts=FAKE, B=1, N=0, pos=None, HQ=8, q=FAKE, qs=1024,
           k=FAKE, ks=256, v=FAKE, vs=256, out=FAKE):
    return lib.gdn_spec_norm_rope_append(ref(p or plan()), ref(qn), ref(kn), ref(c or cache()), layer, slot, starts, B, N, pos,
                                         HQ, q, qs, k, ks, v, vs, out, None)


def rotate(lib, p=None, w=None, N=0, heads=4, io=0, pos=FAKE, x=FAKE, xs=512, out=FAKE + 65536, os_=512):
    return lib.gdn_spec_norm_rope(ref(p or plan()), ref(w or norm()), N, heads, io, pos, x, xs, out, os_, None)


def gradient(lib, p=None, w=None, N=1, heads=4, io=0, pos=FAKE, x=FAKE, xs=512, dy=FAKE, ys=512, dx=FAKE + 65536, ds=512,
             dw=FAKE, ws=FAKE, n=1 << 40):
    return lib.gdn_spec_norm_rope_grad(ref(p or plan()), ref(w or norm()), N, heads, io, pos, x, xs, dy, ys, dx, ds, dw, ws, n,
                                       None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_descriptor(lib, kw, want):
    c = cache(**kw)
    assert attn(lib, c) == want and append(lib, c) == want
    assert lib.gdn_spec_prompt_attn_workspace(ref(c), 1, 4, 8) == want
    assert lib.gdn_spec_prompt_attn_path(ref(c), 8) is None


def test_attention_call(lib):
    c = cache()
    assert attn(lib, c) == OK and attn(lib, c, B=0, N=5) == OK
    for kw, want in ((dict(layer=3), EINVAL), (dict(layer=-1), EINVAL), (dict(B=-1), EINVAL), (dict(N=-1), EINVAL),
                     (dict(HQ=7), EINVAL), (dict(HQ=0), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
                     (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL), (dict(scale=3e38), EINVAL),
                     (dict(N=1, slot=None), EINVAL), (dict(N=1, starts=None), EINVAL), (dict(N=1, q=None), EINVAL),
                     (dict(N=1, out=None), EINVAL), (dict(N=1, ws=None), EINVAL), (dict(N=1, q=MIS), EALIGN),
                     (dict(N=1, out=MIS), EALIGN), (dict(N=1, ws=MIS), EALIGN)):
        assert attn(lib, c, **kw) == want, kw
    assert attn(lib, None) == EINVAL
    assert lib.gdn_spec_prompt_attn_path(ref(c), 8) == b"tc"
    assert lib.gdn_spec_prompt_attn_path(ref(cache(D=96)), 2 * 300) == b"tc"
    assert lib.gdn_spec_prompt_attn_path(ref(cache(io_dtype=1)), 8) == b"generic"
    assert lib.gdn_spec_prompt_attn_path(ref(c), 7) is None and lib.gdn_spec_prompt_attn_path(None, 8) is None


def test_attention_limits(lib):
    text = entry("gdn_spec_prompt_attn -- causal", "int gdn_spec_prompt_attn(")
    assert "HQ / HKV is at most 4096" in text
    assert attn(lib, cache(), HQ=2 * 4096) == OK and attn(lib, cache(), HQ=2 * 4097) == EUNSUP
    assert "n_layers * num_pages * HKV * P is below 2^31" in text
    for io, pages, want in ((0, (1 << 31) // (2 * 64 * 4) - 1, OK), (0, (1 << 31) // (2 * 64 * 4), EUNSUP),
                            (1, (1 << 31) // (2 * 64 * 4), OK)):
        assert attn(lib, cache(n_layers=4, HKV=2, P=64, num_pages=pages, io_dtype=io)) == want
    assert "max_pages * P at most 2^31 - 1025" in text
    for pages, want in (((1 << 31) // 16 - 65, OK), ((1 << 31) // 16 - 64, EUNSUP), ((1 << 31) // 16 - 1, EUNSUP)):
        assert attn(lib, cache(P=16, max_pages=pages)) == want, pages
    assert "(N + B) * HKV * (1 + HQ / HKV / 64) * (max_pages * P + 1024) at most 4e18" in text
    wide = cache(io_dtype=1, P=16, max_pages=(1 << 31) // 16 - 65, HKV=1 << 10)
    assert attn(lib, wide, HQ=1 << 10, B=0, N=1 << 20) == OK and attn(lib, wide, HQ=1 << 10, B=0, N=1 << 21) == EUNSUP


def test_norm(lib):
    for bad, want in ((norm(weight=None), EINVAL), (norm(eps=0.0), EINVAL), (norm(eps=-1.0), EINVAL), (norm(eps=math.nan), EINVAL),
                      (norm(eps=math.inf), EINVAL), (norm(offset=math.nan), EINVAL), (norm(weight=FAKE + 2), EALIGN)):
        assert rotate(lib, w=bad) == want and gradient(lib, w=bad, N=0) == want
        assert append(lib, qn=bad) == want and append(lib, kn=bad) == want
    assert lib.gdn_spec_norm_rope(ref(plan()), None, 0, 4, 0, FAKE, FAKE, 512, FAKE, 512, None) == EINVAL


def test_the_smallest_eps(lib):
    """The gradient forms 1 / (mean(x^2) + eps): for a head of zeros and a small eps that is infinite in fp32, and times zero NaN."""
    least = 2.0 ** -126
    assert "eps;            /* >= 2^-126, finite" in open(HEADER).read()
    assert rotate(lib, w=norm(eps=least)) == OK
    below = norm(eps=least / 2)
    assert 0.0 < below.eps < least
    assert rotate(lib, w=below) == EINVAL and gradient(lib, w=below, N=0) == EINVAL
    assert append(lib, qn=below) == EINVAL and append(lib, kn=below) == EINVAL


def test_rotate_call(lib):
    assert rotate(lib) == OK
    for kw, want in ((dict(N=-1), EINVAL), (dict(heads=0), EINVAL), (dict(io=2), EDTYPE), (dict(xs=511), EINVAL),
                     (dict(xs=513), EALIGN), (dict(os_=516), EALIGN), (dict(N=1, pos=None), EINVAL), (dict(N=1, x=None), EINVAL),
                     (dict(N=1, out=None), EINVAL), (dict(N=1, x=MIS), EALIGN), (dict(N=1, out=MIS), EALIGN),
                     (dict(out=FAKE, os_=520), EINVAL), (dict(heads=1 << 16, xs=1 << 24, os_=1 << 24), EUNSUP)):
        assert rotate(lib, **kw) == want, kw


def test_gradient_call(lib):
    for kw, want in ((dict(N=-1), EINVAL), (dict(heads=0), EINVAL), (dict(io=2), EDTYPE), (dict(xs=511), EINVAL),
                     (dict(ys=511), EINVAL), (dict(ds=511), EINVAL), (dict(ys=513), EALIGN), (dict(dw=None), EINVAL),
                     (dict(dw=MIS), EALIGN), (dict(pos=None), EINVAL), (dict(x=None), EINVAL), (dict(dy=None), EINVAL),
                     (dict(dx=None), EINVAL), (dict(dy=MIS), EALIGN), (dict(ws=MIS), EALIGN), (dict(dx=FAKE, ds=520), EINVAL),
                     (dict(heads=1 << 16, xs=1 << 24, ys=1 << 24, ds=1 << 24), EUNSUP)):
        assert gradient(lib, **kw) == want, kw
    for a, want in (((-1, 4, 128), EINVAL), ((4, 0, 128), EINVAL), ((4, 4, 0), EINVAL), ((4, 4, 100), EALIGN),
                    ((4, 4, 264), EUNSUP), ((4, 1 << 16, 128), EUNSUP)):
        assert lib.gdn_spec_norm_rope_grad_workspace(*a) == want


def test_append_call(lib):
    assert append(lib) == OK and append(lib, qn=norm(), kn=norm()) == OK and append(lib, B=0, N=4) == OK
    for kw, want in ((dict(layer=3), EINVAL), (dict(layer=-1), EINVAL), (dict(B=-1), EINVAL), (dict(N=-1), EINVAL),
                     (dict(HQ=0), EINVAL), (dict(p=plan(64, 64)), EINVAL), (dict(qs=1023), EINVAL), (dict(ks=255), EINVAL),
                     (dict(vs=248), EINVAL), (dict(qs=1028), EALIGN), (dict(ks=260), EALIGN), (dict(vs=260), EALIGN),
                     (dict(N=1, slot=None), EINVAL), (dict(N=1, starts=None), EINVAL), (dict(N=1, q=None), EINVAL),
                     (dict(N=1, k=None), EINVAL), (dict(N=1, v=None), EINVAL), (dict(N=1, out=None), EINVAL),
                     (dict(N=1, q=MIS), EALIGN), (dict(N=1, v=MIS), EALIGN), (dict(N=1, out=MIS), EALIGN),
                     (dict(HQ=1 << 15, qs=1 << 23), EUNSUP)):
        assert append(lib, **kw) == want, kw
    assert "(HQ + 2 HKV) * D is at most 2^22" in entry("gdn_spec_norm_rope_append -- q_out", "int gdn_spec_norm_rope_append(")
    assert append(lib, HQ=(1 << 15) - 4, qs=1 << 22) == OK and append(lib, HQ=(1 << 15) - 3, qs=1 << 22) == EUNSUP


def test_descriptor_mirrors_the_header():
    text = open(HEADER).read()
    body = text[text.index("/* The norm of a head x of D dims"):text.index("} gdn_spec_head_norm;")]
    fields = re.findall(r"^\s+(?:const float \*|float )\s*(\w+);", body, re.M)
    assert fields == [n for n, _ in binding.HeadNormDesc._fields_] and ctypes.sizeof(binding.HeadNormDesc) == 16
