"""Rotary positions and the append to the paged cache against the 64-bit definition.

Bounds: a pair's results are x c - y s and x s + y c with cos and sin to 2^-22 of 1 (the
angle is exact to 2^-32 of a turn and sincospi to two units), so fp32 results are within
2^-21 mscale (|x| + |y|) of the definition, and bf16 ones within half a unit more (eight
significant bits: at most 2^-8 of the result, as the definition rounded to bf16 is).
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu

SCALINGS = [dict(), dict(base=1.0e6), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=32.0, original=4096.0),
            dict(scaling="bands", base=5.0e5, factor=8.0, original=8192.0)]


def close(got, want, x, io, mscale, rot, layout):
    """got against want, elementwise, for pairs of x."""
    i = np.arange(rot // 2)
    i0, i1 = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    size = np.zeros_like(x)
    size[..., i0] = size[..., i1] = (np.abs(x[..., i0]) + np.abs(x[..., i1])) * mscale
    bound = 2.0 ** -21 * size + (2.0 ** -8 if io == "bf16" else 2.0 ** -24) * np.abs(want)
    err = np.abs(got - want)
    assert (err <= bound).all(), np.max(err - bound)
    assert np.array_equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (256, 64), (64, 32), (96, 96), (40, 24), (16, 2), (64, 30), (8, 8)])
@pytest.mark.parametrize("transpose", [False, True])
def test_every_layout_and_part(io, layout, D, rot, transpose):
    rng = np.random.default_rng(1)
    x = ref.draw(rng, (9, 3, D), io)
    pos = np.array([0, 1, 2, 63, 1000, 4097, 131071, 1 << 20, 1999999999], np.int32)
    plan = binding.RopePlan(D, rot, layout=layout, base=1.0e4)
    got = binding.rope(plan, torch.from_numpy(pos).cuda(), x.cuda(), transpose=transpose)
    f, m = ref.frequencies(rot)
    # at 2e9 the definition's own angle is off by 2^-53 of it: 2e-7; the other positions by far less
    x64 = x.double().numpy()
    want = ref.rotate(x64, pos, f, m, rot, layout, transpose)
    close(got[:8].double().cpu().numpy(), want[:8], x64[:8], io, m, rot, layout)
    loose = 4e-2 if io == "bf16" else 2e-6
    assert np.max(np.abs(got[8].double().cpu().numpy() - want[8])) <= loose


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("n", [1, 5, 4099])
def test_scalings_and_many_tokens(kw, n):
    rng = np.random.default_rng(2)
    x = ref.draw(rng, (n, 2, 128), "fp32")
    pos = rng.integers(0, 200000, n).astype(np.int32)
    got = binding.rope(binding.RopePlan(128, 64, **kw), torch.from_numpy(pos).cuda(), x.cuda())
    f, m = ref.frequencies(64, **kw)
    x64 = x.double().numpy()
    close(got.double().cpu().numpy(), ref.rotate(x64, pos, f, m, 64, "half"), x64, "fp32", m, 64, "half")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_transpose_is_the_gradient(layout):
    """<g, R x> against differences: R is linear, so d <g, R x> / dx is R^T g exactly, up to the fp32
    rounding of the two calls (each result within 2^-20 of |x| + |y|)."""
    rng = np.random.default_rng(3)
    plan = binding.RopePlan(64, 48, layout=layout, scaling="yarn", factor=16.0, original=2048.0)
    x, g = (ref.draw(rng, (50, 4, 64), "fp32") for _ in range(2))
    pos = torch.from_numpy(rng.integers(0, 100000, 50).astype(np.int32)).cuda()
    grad = binding.rope(plan, pos, g.cuda(), transpose=True).double().cpu()
    g64 = g.double()
    y = binding.rope(plan, pos, x.cuda()).double().cpu()
    for step in range(6):
        e = torch.zeros_like(x)
        i = rng.integers(0, x.numel())
        e.view(-1)[i] = 1.0
        y2 = binding.rope(plan, pos, (x + e).cuda()).double().cpu()
        slope = float(((y2 - y) * g64).sum() / (float((x + e).view(-1)[i]) - float(x.view(-1)[i])))
        assert abs(slope - float(grad.view(-1)[i])) <= 2e-5
    # and the inner products agree: <g, R x> = <R^T g, x>
    a, b = float((y * g64).sum()), float((grad * x.double()).sum())
    assert abs(a - b) <= 2.0 ** -20 * float((y.abs() * g64.abs()).sum())


def test_in_place_strides_and_empty():
    rng = np.random.default_rng(4)
    wide = ref.draw(rng, (37, 6, 128), "bf16").cuda()
    keep = wide.clone()
    pos = torch.arange(37, dtype=torch.int32, device="cuda")
    plan = binding.RopePlan(128)
    part = wide[:, 1:4]
    want = binding.rope(plan, pos, part.contiguous())
    assert torch.equal(binding.rope(plan, pos, part), want)
    binding.rope(plan, pos, part, out=part)
    assert torch.equal(part, want) and torch.equal(wide[:, 0], keep[:, 0]) and torch.equal(wide[:, 4:], keep[:, 4:])
    assert binding.rope(plan, pos[:0], part[:0]).shape == (0, 3, 128)
    with pytest.raises(binding.GdnSpecError):
        binding.rope(plan, pos, wide[:, :, :64])
    with pytest.raises(binding.GdnSpecError):
        binding.rope(plan, pos[:3], part)
    with pytest.raises(binding.GdnSpecError):
        binding.rope(plan, pos, part.half())
    with pytest.raises(binding.GdnSpecError):
        binding.rope(plan, pos, wide[:, ::2])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T,HQ,HKV,D,rot,P,layout", [
    (1, 4, 2, 128, 128, 16, "half"), (8, 16, 2, 256, 64, 64, "half"), (5, 3, 3, 64, 64, 32, "interleaved"),
    (40, 2, 1, 40, 20, 16, "interleaved"), (2100, 2, 1, 64, 32, 128, "half"), (7, 6, 2, 48, 24, 256, "half")])
@pytest.mark.parametrize("given", [False, True])
def test_append(io, T, HQ, HKV, D, rot, P, layout, given):
    """Slices of one projection, ragged counts, a padding row; nothing but the window's rows is written."""
    rng = np.random.default_rng(5)
    lens = np.array([0, 3 * P - 1, P, 29, 70], np.int32)
    slots = np.array([0, 1, -1, 4, 3], np.int32)
    B = len(slots)
    counts = np.array([T, max(1, T // 2), T, T, 0], np.int32)
    pages = sum(-(-(int(n) + T) // P) for n in lens) + 1
    max_pages = max(-(-(int(n) + T) // P) for n in lens)
    table, count = ref.pages_for(rng, lens, T, P, pages, max_pages)
    shape = (2, pages, HKV, P, D)
    k0, v0 = ref.draw(rng, shape, io), ref.draw(rng, shape, io)
    cache = binding.KvCache(2, pages, HKV, P, D, len(lens), max_pages, io, tensors={
        "k": k0.cuda(), "v": v0.cuda(), "page_table": torch.from_numpy(table).cuda(),
        "n_pages": torch.from_numpy(count).cuda(), "length": torch.from_numpy(lens).cuda()})
    qkv = ref.draw(rng, (B, T, HQ + 2 * HKV, D), io)
    dev = qkv.cuda()
    pos = rng.integers(0, 50000, (B, T)).astype(np.int32)
    if not given:
        pos = np.array([lens[s] + np.arange(T) if s >= 0 else np.zeros(T) for s in slots]).astype(np.int32)
    plan = binding.RopePlan(D, rot, layout=layout, scaling="bands", base=1.0e5, factor=4.0, original=1000.0)
    out = binding.rope_append(plan, cache, 1, torch.from_numpy(slots).cuda(), dev[:, :, :HQ],
                              dev[:, :, HQ:HQ + HKV], dev[:, :, HQ + HKV:],
                              pos=torch.from_numpy(pos).cuda() if given else None,
                              n_tokens=torch.from_numpy(counts).cuda())
    assert binding.kv_read_status(cache) == 0
    f, m = ref.frequencies(rot, base=1.0e5, scaling="bands", factor=4.0, original=1000.0)
    x = qkv.double().numpy()
    turned = ref.rotate(x[:, :, :HQ + HKV], pos, f, m, rot, layout)
    got = out.double().cpu().numpy()
    kg, vg = cache.k.cpu(), cache.v.cpu()
    k1, v1 = k0.clone(), v0.clone()
    for b, s in enumerate(slots):
        n = int(counts[b]) if s >= 0 else 0
        assert (got[b, n:] == 0).all()
        if not n:
            continue
        close(got[b, :n], turned[b, :n, :HQ], x[b, :n, :HQ], io, m, rot, layout)
        i = int(lens[s]) + np.arange(n)
        page, off = torch.from_numpy(table[s, i // P]).long(), torch.from_numpy(i % P)
        close(kg[1, page, :, off].double().numpy(), turned[b, :n, HQ:], x[b, :n, HQ:HQ + HKV], io, m, rot, layout)
        k1[1, page, :, off] = kg[1, page, :, off]
        v1[1, page, :, off] = qkv[b, :n, HQ + HKV:]
    assert torch.equal(kg, k1) and torch.equal(vg, v1)


def test_append_refusals():
    cache = binding.KvCache(1, 8, 2, 16, 64, 4, 4, "bf16")
    cache.k.zero_(), cache.v.zero_()
    slots = torch.tensor([0, 1, 2, 7], dtype=torch.int32, device="cuda")
    binding.kv_reserve(cache, slots[:3], 16)
    cache.n_pages[1] = 0                                  # no pages
    cache.page_table[2, 0] = 99
    plan = binding.RopePlan(64)
    qkv = torch.ones(4, 3, 8, 64, dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    out = binding.rope_append(plan, cache, 0, slots, q, k, v)
    assert binding.kv_read_status(cache) == binding.ST_NO_PAGES | binding.ST_SLOT_OOR | binding.ST_PAGE_OOR
    assert (out[1:] == 0).all() and (out[0] != 0).any()
    assert int((cache.v != 0).any(-1).sum()) == 3 * 2     # the first row's tokens, two heads
    cnt = torch.tensor([4, 0, 0, 0], dtype=torch.int32, device="cuda")
    out = binding.rope_append(plan, cache, 0, slots[:1], q[:1], k[:1], v[:1], n_tokens=cnt[:1])
    assert binding.kv_read_status(cache) == binding.ST_ACCEPT_RANGE and (out == 0).all()
    for bad in (lambda: binding.rope_append(plan, cache, 1, slots, q, k, v),
                lambda: binding.rope_append(binding.RopePlan(128), cache, 0, slots, q, k, v),
                lambda: binding.rope_append(plan, cache, 0, slots, q, k[:, :, :1], v),
                lambda: binding.rope_append(plan, cache, 0, slots, q.float(), k, v),
                lambda: binding.rope_append(plan, cache, 0, slots, q.transpose(1, 2), k, v)):
        with pytest.raises(binding.GdnSpecError):
            bad()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,D,rot", [(33001, 1, 64, 64), (17003, 2, 128, 48), (33005, 1, 40, 24), (16387, 3, 256, 256)])
def test_many_tokens_of_few_heads(io, layout, n, heads, D, rot):
    """Blocks of eight and sixteen tokens, the last one short."""
    rng = np.random.default_rng(6)
    x = ref.draw(rng, (n, heads, D), io)
    pos = rng.integers(0, 200000, n).astype(np.int32)
    got = binding.rope(binding.RopePlan(D, rot, layout=layout), torch.from_numpy(pos).cuda(), x.cuda())
    f, m = ref.frequencies(rot)
    x64 = x.double().numpy()
    close(got.double().cpu().numpy(), ref.rotate(x64, pos, f, m, rot, layout), x64, io, m, rot, layout)


@pytest.mark.parametrize("io,T,HQ,HKV,D,rot,P,layout", [
    ("bf16", 6700, 1, 1, 32, 16, 128, "half"), ("fp32", 4100, 2, 1, 64, 64, 64, "interleaved"),
    ("bf16", 6601, 1, 1, 24, 20, 32, "interleaved")])
def test_append_many_tokens_of_few_heads(io, T, HQ, HKV, D, rot, P, layout):
    test_append(io, T, HQ, HKV, D, rot, P, layout, False)
