"""Host-side checks of the softmax-attention layers' entry points and the rotary plan,
without a GPU: every call here fails validation or has nothing to do, so the fake
(aligned, never dereferenced) device pointers are never used."""
import ctypes
import math

import pytest

from gated_delta_rule_spec_gb300 import binding
from gated_delta_rule_spec_gb300 import build as lib_build
from tests import attn_ref as ref

OK, EINVAL, EDTYPE, EALIGN, EUNSUP = 0, -1, -2, -3, -5
FAKE = 0x7F0000100000
MIS = FAKE + 8


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return binding.load()


def cache(**kw):
    f = dict(n_layers=3, num_pages=64, HKV=2, P=64, D=128, io_dtype=binding.DTYPE_BF16, num_slots=8, max_pages=16,
             k=FAKE, v=FAKE, page_table=FAKE, n_pages=FAKE, length=FAKE, ref=FAKE, free_bits=FAKE, status=FAKE)
    f.update(kw)
    return binding.KvCacheDesc(*(f[n] for n, _ in binding.KvCacheDesc._fields_))


def attn(lib, c, layer=0, slot=FAKE, B=0, T=4, HQ=8, q=FAKE, scale=0.1, out=FAKE, ws=FAKE, n=1 << 40):
    return lib.gdn_spec_tree_attn(ctypes.byref(c), layer, slot, B, T, HQ, q, None, None, scale, out, None, ws, n, None)


BAD_CACHES = [
    (dict(io_dtype=3), EDTYPE), (dict(n_layers=0), EINVAL), (dict(num_pages=-1), EINVAL), (dict(HKV=0), EINVAL),
    (dict(P=48), EINVAL), (dict(P=8), EUNSUP), (dict(P=512), EUNSUP), (dict(D=100), EALIGN), (dict(D=264), EUNSUP),
    (dict(num_slots=0), EINVAL), (dict(max_pages=0), EINVAL), (dict(k=None), EINVAL), (dict(status=None), EINVAL),
    (dict(free_bits=None), EINVAL), (dict(v=MIS), EALIGN), (dict(num_pages=1 << 25, P=64), EUNSUP),
    (dict(max_pages=1 << 26), EUNSUP)]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_descriptor(lib, kw, want):
    c = cache(**kw)
    r = ctypes.byref(c)
    assert lib.gdn_spec_kv_init(r, None) == want
    assert lib.gdn_spec_kv_reserve(r, FAKE, 0, 4, None, FAKE, None) == want
    assert lib.gdn_spec_kv_fork(r, FAKE, FAKE, 0, FAKE, None) == want
    assert lib.gdn_spec_kv_commit(r, FAKE, 0, 4, None, FAKE, None) == want
    assert lib.gdn_spec_kv_free(r, FAKE, 0, None) == want
    assert lib.gdn_spec_kv_read_status(r, ctypes.byref(ctypes.c_uint32()), 0, None) == want
    assert attn(lib, c) == want
    assert lib.gdn_spec_tree_attn_workspace(r, 1, 4, 8) == want
    assert lib.gdn_spec_tree_attn_path(r, 4, 8) is None


def test_null_descriptors(lib):
    assert lib.gdn_spec_kv_init(None, None) == EINVAL
    assert lib.gdn_spec_tree_attn(None, 0, FAKE, 0, 4, 8, FAKE, None, None, 1.0, FAKE, None, FAKE, 0, None) == EINVAL
    assert lib.gdn_spec_tree_attn_path(None, 4, 8) is None
    assert lib.gdn_spec_kv_read_status(ctypes.byref(cache()), None, 0, None) == EINVAL


def test_page_calls(lib):
    r = ctypes.byref(cache())
    assert lib.gdn_spec_kv_reserve(r, FAKE, 0, 4, None, FAKE, None) == OK
    assert lib.gdn_spec_kv_reserve(r, FAKE, -1, 4, None, FAKE, None) == EINVAL
    assert lib.gdn_spec_kv_reserve(r, FAKE, 1, -4, None, FAKE, None) == EINVAL
    assert lib.gdn_spec_kv_reserve(r, None, 1, 4, None, FAKE, None) == EINVAL
    assert lib.gdn_spec_kv_reserve(r, FAKE, 1, 4, None, None, None) == EINVAL
    assert lib.gdn_spec_kv_reserve(r, FAKE, 8193, 4, None, FAKE, None) == EUNSUP
    assert lib.gdn_spec_kv_fork(r, FAKE, FAKE, 0, FAKE, None) == OK
    assert lib.gdn_spec_kv_fork(r, FAKE, None, 1, FAKE, None) == EINVAL
    assert lib.gdn_spec_kv_fork(r, FAKE, FAKE, -2, FAKE, None) == EINVAL
    assert lib.gdn_spec_kv_fork(r, FAKE, FAKE, 9000, FAKE, None) == EUNSUP
    assert lib.gdn_spec_kv_commit(r, FAKE, 0, 4, None, FAKE, None) == OK
    assert lib.gdn_spec_kv_commit(r, FAKE, 1, 0, None, FAKE, None) == EINVAL
    assert lib.gdn_spec_kv_commit(r, FAKE, 1, 4, None, None, None) == EINVAL
    assert lib.gdn_spec_kv_commit(r, FAKE, 1, 1025, FAKE, FAKE, None) == EUNSUP
    assert lib.gdn_spec_kv_free(r, FAKE, 0, None) == OK
    assert lib.gdn_spec_kv_free(r, None, 1, None) == EINVAL


def test_attention_call(lib):
    c = cache()
    assert attn(lib, c) == OK
    for kw, want in ((dict(layer=3), EINVAL), (dict(layer=-1), EINVAL), (dict(B=-1), EINVAL), (dict(T=0), EINVAL),
                     (dict(T=65), EUNSUP), (dict(HQ=7), EINVAL), (dict(HQ=0), EINVAL), (dict(scale=0.0), EINVAL),
                     (dict(scale=-1.0), EINVAL), (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL),
                     (dict(B=1, slot=None), EINVAL), (dict(B=1, q=None), EINVAL), (dict(B=1, out=MIS), EALIGN),
                     (dict(B=1, ws=None), EINVAL), (dict(B=1, ws=MIS), EALIGN), (dict(HQ=2 * 4097), EUNSUP)):
        assert attn(lib, c, **kw) == want, kw
    assert lib.gdn_spec_tree_attn_path(ctypes.byref(c), 65, 8) is None
    assert lib.gdn_spec_tree_attn_path(ctypes.byref(cache(io_dtype=1)), 4, 8) == b"generic"
    assert lib.gdn_spec_tree_attn_path(ctypes.byref(cache(D=96)), 4, 8) == b"tc"
    assert lib.gdn_spec_tree_attn_path(ctypes.byref(cache()), 4, 2 * 129) == b"generic"


def test_attention_counts_in_31_bits(lib):
    short = cache(HKV=1, P=16, max_pages=1)
    assert attn(lib, short, B=1 << 25, T=64) == EUNSUP          # tokens
    assert attn(lib, short, B=(1 << 31) - 1, T=1) == EUNSUP     # tiles: one of 16 tokens is a tile too
    assert attn(lib, cache(max_pages=1 << 20), B=1 << 12) == EUNSUP
    assert lib.gdn_spec_tree_attn_workspace(ctypes.byref(short), 1 << 25, 64, 8) == EUNSUP


def plan(D=128, rot=128, layout="half", **kw):
    return binding.RopePlan(D, rot, layout=layout, **kw).desc()


def test_rope_calls(lib):
    p, c = plan(), cache()

    def rope(N=0, heads=4, io=0, pos=FAKE, x=FAKE, xs=512, out=FAKE + 65536, os_=512, p=p):
        return lib.gdn_spec_rope(ctypes.byref(p), N, heads, io, pos, x, xs, out, os_, 0, None)

    assert rope() == OK
    for kw, want in ((dict(N=-1), EINVAL), (dict(heads=0), EINVAL), (dict(io=2), EDTYPE), (dict(xs=511), EINVAL),
                     (dict(xs=513), EALIGN), (dict(os_=516), EALIGN), (dict(N=1, pos=None), EINVAL),
                     (dict(N=1, x=MIS), EALIGN), (dict(N=1, x=FAKE, out=FAKE, os_=1024), EINVAL)):
        assert rope(**kw) == want, kw
    bad = plan()
    bad.rot = 130
    assert rope(p=bad) == EINVAL
    bad.rot, bad.layout = 64, 5
    assert rope(p=bad) == EINVAL

    def append(p=p, c=c, layer=0, B=0, T=4, HQ=8, q=FAKE, qs=1536, ks=1536, vs=1536, slot=FAKE):
        return lib.gdn_spec_rope_append(ctypes.byref(p), ctypes.byref(c), layer, slot, B, T, None, None, HQ, q, qs,
                                        FAKE, ks, FAKE, vs, FAKE, None)

    assert append() == OK
    for kw, want in ((dict(layer=3), EINVAL), (dict(T=0), EINVAL), (dict(B=-1), EINVAL), (dict(HQ=0), EINVAL),
                     (dict(qs=1016), EINVAL), (dict(ks=248), EINVAL), (dict(vs=1540), EALIGN), (dict(p=plan(64, 64)), EINVAL),
                     (dict(B=1, q=None), EINVAL), (dict(B=1, q=MIS), EALIGN), (dict(B=1, slot=None), EINVAL),
                     (dict(c=cache(P=48)), EINVAL)):
        assert append(**kw) == want, kw


@pytest.mark.parametrize("kw", [dict(), dict(base=1e6), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=32.0, original=4096.0),
                                dict(scaling="yarn", factor=4.0, original=100.0, fast=8.0, slow=2.0),
                                dict(scaling="bands", base=5e5, factor=8.0, original=8192.0),
                                dict(scaling="bands", factor=2.0, original=64.0, low=0.5, high=2.0)])
@pytest.mark.parametrize("rot", [4, 64, 126, 256])
def test_plan_frequencies(lib, kw, rot):
    """Turns per position: the definition's, to the 2^-50 that double arithmetic leaves."""
    d = plan(256, rot, **kw)
    f, m = ref.frequencies(rot, **kw)
    assert d.mscale == ctypes.c_float(m).value
    for i, x in enumerate(f):
        turns = d.freq[i] / 2.0 ** 64
        assert abs(turns - x / (2 * math.pi)) <= 2.0 ** -50 * max(turns, 2.0 ** -14), i
    assert all(d.freq[i] == 0 for i in range(rot // 2, 128))


def test_plan_from_frequencies_and_refusals(lib):
    d = plan(64, 8, freqs=[0.0, 2 * math.pi, -math.pi / 2, 1e-9], mscale=0.5)
    assert d.mscale == 0.5 and d.freq[0] == 0
    assert d.freq[1] == 0 and d.freq[2] == 3 << 62            # whole turns fall away, negative ones wrap
    assert abs(d.freq[3] / 2.0 ** 64 - 1e-9 / (2 * math.pi)) <= 2.0 ** -64   # the format's unit
    for kw in (dict(rot=0), dict(rot=3), dict(rot=130), dict(D=100, rot=20), dict(layout="odd"), dict(scaling="odd"),
               dict(base=1.0), dict(base=math.nan), dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=2.0),
               dict(scaling="yarn", factor=2.0, original=10.0, fast=1.0, slow=2.0), dict(rot=2, scaling="ntk", factor=2.0),
               dict(scaling="bands", factor=2.0, original=10.0, low=4.0, high=4.0), dict(freqs=[1.0]),
               dict(freqs=[math.inf] * 64), dict(mscale=math.nan, freqs=[1.0] * 64)):
        with pytest.raises(binding.GdnSpecError):
            plan(**kw)


def test_descriptor_layouts():
    assert ctypes.sizeof(binding.KvCacheDesc) == 8 * 4 + 8 * 8
    assert ctypes.sizeof(binding.RopePlanDesc) == 16 + 128 * 8
    assert ctypes.sizeof(binding.RopeScalingDesc) == 8 + 4 * 8


def test_constants_match_the_header():
    from tests.test_abi_exports import _header_defines
    d = _header_defines()
    for name in ("ST_NO_PAGES", "ST_PAGE_OOR", "ST_SLOT_BUSY", "ROPE_HALF", "ROPE_INTERLEAVED", "ROPE_NONE",
                 "ROPE_LINEAR", "ROPE_NTK", "ROPE_YARN", "ROPE_BANDS"):
        assert d["GDN_SPEC_" + name] == getattr(binding, name)
