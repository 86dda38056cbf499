"""The heads' norm with its rotary position, its append to the cache and its gradient against the 64-bit
definitions.

Bounds: the sum of D <= 256 squares is of 16 terms in a thread and of at most 16 threads in a
tree (or 16 in a lane and 32 lanes), each addition off by 2^-24 of the sum, so it is within 2^-19 of itself
and the root within 2^-20, plus two units of rsqrt; cos and sin are within 2^-22; with the few
products a result is within 2^-18 of the size of its terms, plus half a unit of its type (2^-8,
2^-24).  dx likewise with its second sum: 2^-17.  dw is a sum of up to some 200 terms in a thread
(2^-16.3) and of the threads and blocks in trees and runs of at most 20: 2^-15.5 of the terms' size in all.
"""
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests import attn_ref as ref
from tests import norm_ref
from tests.prompt_case import Prompts

pytestmark = pytest.mark.gpu

HALF_ULP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
SHAPES = [(128, 128), (256, 64), (64, 32), (96, 96), (96, 48), (40, 24), (16, 2), (64, 30), (8, 8), (16, 16), (200, 20),
          (256, 256), (32, 32), (208, 16)]
YARN = dict(scaling="yarn", base=1.0e4, factor=16.0, original=2048.0)


def weights(rng, D, offset):
    return torch.from_numpy((1.0 - offset + 0.3 * rng.standard_normal(D)).astype(np.float32))


def close(got, want, terms, io, noise=2.0 ** -18):
    err, bound = np.abs(got - want), noise * terms + HALF_ULP[io] * np.abs(want)
    assert np.isfinite(got).all() and (err <= bound).all(), np.max(err - bound)


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", SHAPES)
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_every_layout_and_part(io, layout, D, rot, offset):
    rng = np.random.default_rng(1)
    x = ref.draw(rng, (9, 3, D), io) * 3
    x[4, 1] = 0                                           # a head of zeros
    x[5, 0] *= 1e-4                                       # one beside which eps counts
    pos = np.array([0, 1, 2, 63, 1000, 4097, 131071, 1 << 20, 7], np.int32)
    w = weights(rng, D, offset)
    plan = binding.RopePlan(D, rot, layout=layout, **(YARN if rot > 8 else {}))
    got = binding.norm_rope(plan, binding.HeadNorm(w.cuda(), eps=1e-5, offset=offset), torch.from_numpy(pos).cuda(), x.cuda())
    f, m = ref.frequencies(rot, **(YARN if rot > 8 else {}))
    x64, w64 = x.double().numpy(), w.double().numpy() + offset
    y = x64 * norm_ref.root(x64, np.float64(np.float32(1e-5))) * w64
    close(got.double().cpu().numpy(), ref.rotate(y, pos, f, m, rot, layout), norm_ref.size(y, rot, layout, m), io)
    assert (got[4, 1] == 0).all()


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,D,rot", [(1, 16, 128, 128), (33001, 1, 64, 64), (17003, 2, 128, 48), (33005, 1, 40, 24),
                                           (5000, 5, 96, 48), (4099, 16, 256, 64), (1, 1, 16, 16), (2, 7, 80, 40)])
def test_token_counts(io, layout, n, heads, D, rot):
    """Blocks of one to sixteen tokens, the last one short; and the gradient of the same tensors."""
    rng = np.random.default_rng(2)
    x, dy = (ref.draw(rng, (n, heads, D), io) for _ in range(2))
    pos = rng.integers(0, 200000, n).astype(np.int32)
    w = weights(rng, D, 0.0)
    plan, norm, p = binding.RopePlan(D, rot, layout=layout), binding.HeadNorm(w.cuda()), torch.from_numpy(pos).cuda()
    got = binding.norm_rope(plan, norm, p, x.cuda())
    f, m = ref.frequencies(rot)
    x64, w64, eps = x.double().numpy(), w.double().numpy(), np.float64(np.float32(1e-6))
    y = x64 * norm_ref.root(x64, eps) * w64
    close(got.double().cpu().numpy(), ref.rotate(y, pos, f, m, rot, layout), norm_ref.size(y, rot, layout, m), io)
    dx, dw = binding.norm_rope_grad(plan, norm, p, x.cuda(), dy.cuda())
    wx, ww, sx, sw = norm_ref.gradient(x64, dy.double().numpy(), w64, eps, pos, f, m, rot, layout)
    close(dx.double().cpu().numpy(), wx, sx, io, 2.0 ** -17)
    close(dw.double().cpu().numpy(), ww, sw, "fp32", 2.0 ** -15.5)


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", SHAPES)
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_gradient(io, layout, D, rot, offset):
    rng = np.random.default_rng(3)
    x, dy = (ref.draw(rng, (50, 3, D), io) for _ in range(2))
    x[4, 1] = 0
    pos = rng.integers(0, 100000, 50).astype(np.int32)
    w = weights(rng, D, offset)
    plan = binding.RopePlan(D, rot, layout=layout, **(YARN if rot > 8 else {}))
    norm = binding.HeadNorm(w.cuda(), eps=1e-4, offset=offset)
    dx, dw = binding.norm_rope_grad(plan, norm, torch.from_numpy(pos).cuda(), x.cuda(), dy.cuda())
    f, m = ref.frequencies(rot, **(YARN if rot > 8 else {}))
    wx, ww, sx, sw = norm_ref.gradient(x.double().numpy(), dy.double().numpy(), w.double().numpy() + offset,
                                       np.float64(np.float32(1e-4)), pos, f, m, rot, layout)
    close(dx.double().cpu().numpy(), wx, sx, io, 2.0 ** -17)
    close(dw.double().cpu().numpy(), ww, sw, "fp32", 2.0 ** -15.5)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 48), (40, 24)])
def test_gradient_against_differences(layout, D, rot):
    """<g, y(x)> and <g, y(w)> by central differences of the forward call: steps of 2^-5 leave h^2 / 6 = 1.6e-4 of the third
    derivative (below 10: heads of root mean square one) and the two calls' rounding, 2^-18 of some sqrt(D) terms
    below 4 over 2^-4: 2e-3 in all."""
    rng = np.random.default_rng(4)
    x, g = (ref.draw(rng, (5, 2, D), "fp32") for _ in range(2))
    pos = torch.from_numpy(rng.integers(0, 1000, 5).astype(np.int32)).cuda()
    w = weights(rng, D, 0.0)
    plan, h = binding.RopePlan(D, rot, layout=layout), 2.0 ** -5
    loss = lambda x, w: float((binding.norm_rope(plan, binding.HeadNorm(w.cuda()), pos, x.cuda()).double().cpu()  # noqa: E731
                               * g.double()).sum())
    dx, dw = (t.double().cpu() for t in binding.norm_rope_grad(plan, binding.HeadNorm(w.cuda()), pos, x.cuda(), g.cuda()))
    for _ in range(8):
        i, e = int(rng.integers(0, x.numel())), torch.zeros_like(x)
        e.view(-1)[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - float(dx.view(-1)[i])) <= 2e-3
        i, e = int(rng.integers(0, D)), torch.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - float(dw[i])) <= 2e-3


def test_in_place_strides_and_empty():
    rng = np.random.default_rng(5)
    wide, dwide = (ref.draw(rng, (37, 6, 128), "bf16").cuda() for _ in range(2))
    keep = wide.clone()
    pos = torch.arange(37, dtype=torch.int32, device="cuda")
    plan, norm = binding.RopePlan(128), binding.HeadNorm(weights(rng, 128, 1.0).cuda(), offset=1.0)
    part, dpart = wide[:, 1:4], dwide[:, 2:5]
    want = binding.norm_rope(plan, norm, pos, part.contiguous())
    wx, ww = binding.norm_rope_grad(plan, norm, pos, part.contiguous(), dpart.contiguous())
    assert torch.equal(binding.norm_rope(plan, norm, pos, part), want)
    dx, dw = binding.norm_rope_grad(plan, norm, pos, part, dpart)
    assert torch.equal(dx, wx) and torch.equal(dw, ww)
    for over in ("dy", "x"):
        a, b = wide.clone(), dwide.clone()
        place = b[:, 2:5] if over == "dy" else a[:, 1:4]
        out = binding.norm_rope_grad(plan, norm, pos, a[:, 1:4], b[:, 2:5], dx=place)
        assert torch.equal(place, wx) and torch.equal(out[1], ww)
    binding.norm_rope(plan, norm, pos, part, out=part)
    assert torch.equal(part, want) and torch.equal(wide[:, 0], keep[:, 0]) and torch.equal(wide[:, 4:], keep[:, 4:])
    assert binding.norm_rope(plan, norm, pos[:0], part[:0]).shape == (0, 3, 128)
    dw = torch.full((128,), 7.0, device="cuda")
    binding.norm_rope_grad(plan, norm, pos[:0], part[:0], dpart[:0], dw=dw)
    assert (dw == 0).all()


def test_gradient_repeats_in_a_graph_and_on_a_stream():
    """The same bits from every call, also captured, replayed and on another stream; the workspace may hold anything."""
    rng = np.random.default_rng(6)
    x, dy = (ref.draw(rng, (6001, 4, 128), "bf16").cuda() for _ in range(2))
    pos = torch.arange(6001, dtype=torch.int32, device="cuda")
    plan, norm = binding.RopePlan(128), binding.HeadNorm(weights(rng, 128, 0.0).cuda())
    dx, dw = binding.norm_rope_grad(plan, norm, pos, x, dy)
    work = torch.full((binding.norm_rope_grad_workspace(6001, 4, 128),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(10):
        a, b = binding.norm_rope_grad(plan, norm, pos, x, dy, workspace=work)
        assert torch.equal(a, dx) and torch.equal(b, dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = binding.norm_rope_grad(plan, norm, pos, x, dy, stream=s)
    s.synchronize()
    assert torch.equal(a, dx) and torch.equal(b, dw)
    g, a, b = torch.cuda.CUDAGraph(), torch.zeros_like(dx), torch.zeros_like(dw)
    with torch.cuda.graph(g):
        binding.norm_rope_grad(plan, norm, pos, x, dy, dx=a, dw=b, workspace=work)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, dx) and torch.equal(b, dw)


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("HQ,HKV,D,rot,P,layout,counts", [
    (4, 2, 128, 128, 16, "half", [1, 1, 1, 1, 1]), (16, 2, 256, 64, 64, "half", [8, 1, 3, 0, 70]),
    (3, 3, 64, 64, 32, "interleaved", [5, 0, 0, 31, 200]), (2, 1, 40, 20, 16, "interleaved", [40, 1, 17, 3, 9]),
    (5, 1, 96, 48, 128, "half", [700, 4000, 13, 1, 0]), (6, 2, 48, 24, 256, "half", [7, 7, 7, 7, 7])])
@pytest.mark.parametrize("given,normed", [(False, "qk"), (True, "qk"), (True, "k"), (False, "")])
def test_append(io, HQ, HKV, D, rot, P, layout, counts, given, normed):
    """Slices of one projection, ragged counts, a padding row, tokens of no row; nothing but the rows' tokens is written."""
    lens = [0, 3 * P - 1, P, 29, 70]
    c = Prompts(7, io, HQ, HKV, D, P, counts, lens, slots=[0, 1, -1, 4, 3], layers=2, layer=1, poison=False, lead=2, tail=3)
    cache, rng = c.upload(), c.rng
    qkv = ref.draw(rng, (c.N, HQ + 2 * HKV, D), io)
    dev = qkv.cuda()
    pos = rng.integers(0, 50000, c.N).astype(np.int32)
    for b, s in enumerate(c.slots):
        if s >= 0 and not given:
            pos[c.starts[b]:c.starts[b + 1]] = lens[s] + np.arange(counts[b])
    kw = dict(scaling="bands", base=1.0e5, factor=4.0, original=1000.0)
    wq, wk = weights(rng, D, 0.0), weights(rng, D, 1.0)
    out = torch.full((c.N, HQ, D), 7.0, dtype=ref.TORCH[io], device="cuda")
    binding.norm_rope_append(
        binding.RopePlan(D, rot, layout=layout, **kw), cache, 1, torch.from_numpy(c.slots).cuda(),
        torch.from_numpy(c.starts).cuda(), dev[:, :HQ], dev[:, HQ:HQ + HKV], dev[:, HQ + HKV:],
        q_norm=binding.HeadNorm(wq.cuda(), eps=1e-5) if "q" in normed else None,
        k_norm=binding.HeadNorm(wk.cuda(), eps=1e-3, offset=1.0) if "k" in normed else None,
        pos=torch.from_numpy(pos).cuda() if given else None, q_out=out)
    assert binding.kv_read_status(cache) == 0
    f, m = ref.frequencies(rot, **kw)
    x = qkv.double().numpy()
    y = x[:, :HQ + HKV].copy()
    if "q" in normed:
        y[:, :HQ] *= norm_ref.root(y[:, :HQ], np.float64(np.float32(1e-5))) * wq.double().numpy()
    if "k" in normed:
        y[:, HQ:] *= norm_ref.root(y[:, HQ:], np.float64(np.float32(1e-3))) * (wk.double().numpy() + 1.0)
    turned, terms = ref.rotate(y, pos, f, m, rot, layout), norm_ref.size(y, rot, layout, m)
    got, kg, vg = out.double().cpu().numpy(), cache.k.cpu(), cache.v.cpu()
    k1, v1 = c.k.clone(), c.v.clone()
    assert (got[:2] == 7).all() and (got[-3:] == 7).all()
    for b, s in enumerate(c.slots):
        a, e = int(c.starts[b]), int(c.starts[b + 1])
        if s < 0:
            assert (got[a:e] == 0).all()
            continue
        if a == e:
            continue
        close(got[a:e], turned[a:e, :HQ], terms[a:e, :HQ], io)
        i = lens[s] + np.arange(e - a)
        page, off = torch.from_numpy(c.table[s, i // P]).long(), torch.from_numpy(i % P)
        close(kg[1, page, :, off].double().numpy(), turned[a:e, HQ:], terms[a:e, HQ:], io)
        k1[1, page, :, off] = kg[1, page, :, off]
        v1[1, page, :, off] = qkv[a:e, HQ + HKV:]
    assert torch.equal(kg, k1) and torch.equal(vg, v1)


@pytest.mark.parametrize("D", [64, 40])
def test_append_refusals(D):
    c = Prompts(8, "bf16", 4, 2, D, 16, [3, 3, 3, 3, 3], [20, 0, 5, 40, 2], slots=[0, 9, 2, 3, 4], poison=False)
    cache = c.upload()
    cache.k.zero_(), cache.v.zero_()
    cache.length[2] = -4
    cache.n_pages[3] = 2                                  # 40 tokens do not fit in two pages of 16
    cache.page_table[4, 0] = 99
    plan, norm = binding.RopePlan(D), binding.HeadNorm(torch.ones(D, device="cuda"))
    qkv = torch.ones(c.N, 8, D, dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    slots, starts = torch.from_numpy(c.slots).cuda(), torch.from_numpy(c.starts).cuda()
    out = binding.norm_rope_append(plan, cache, 0, slots, starts, q, k, v, norm, norm)
    assert binding.kv_read_status(cache) == binding.ST_SLOT_OOR | binding.ST_CURSOR_CORRUPT | binding.ST_PAGE_OOR
    assert (out[3:] == 0).all() and (out[:3] != 0).any()
    assert int((cache.v != 0).any(-1).sum()) == 3 * 2     # the first row's tokens, two heads
    cache.length[3] = 30                                  # 32 rows: the third of them has no place
    binding.norm_rope_append(plan, cache, 0, slots, starts, q, k, v, norm, norm)
    assert binding.kv_read_status(cache) & binding.ST_NO_PAGES
    for bad in ([0, 3, 6, 9, 12, 16], [-1, 3, 6, 9, 12, 15], [0, 3, 6, 9, 12, 10]):
        out = torch.full((c.N, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
        st = torch.tensor(bad, dtype=torch.int32, device="cuda")
        binding.norm_rope_append(plan, cache, 0, slots, st, q, k, v, norm, norm, q_out=out)
        assert binding.kv_read_status(cache) & binding.ST_ACCEPT_RANGE
        mine = slice(0, 3) if bad[0] < 0 else slice(12, 15)
        assert (out[mine] == 7).all()
    two = binding.RopePlan(128)
    for call in (lambda: binding.norm_rope_append(plan, cache, 1, slots, starts, q, k, v),
                 lambda: binding.norm_rope_append(two, cache, 0, slots, starts, q, k, v),
                 lambda: binding.norm_rope_append(plan, cache, 0, slots, starts[:-1], q, k, v),
                 lambda: binding.norm_rope_append(plan, cache, 0, slots, starts, q, k[:, :1], v),
                 lambda: binding.norm_rope_append(plan, cache, 0, slots, starts, q.float(), k, v),
                 lambda: binding.norm_rope_append(plan, cache, 0, slots, starts, q[None], k, v),
                 lambda: binding.norm_rope_append(plan, cache, 0, slots, starts, q, k, v, pos=starts),
                 lambda: binding.norm_rope_append(plan, cache, 0, slots, starts, q, k, v, q_norm=binding.HeadNorm(
                     torch.ones(128, device="cuda"))),
                 lambda: binding.norm_rope_append(plan, cache, 0, slots, starts, q, k, v, q_norm=binding.HeadNorm(
                     torch.ones(D, device="cuda"), eps=0.0))):
        with pytest.raises(binding.GdnSpecError):
            call()


def test_binding_refuses():
    plan, pos = binding.RopePlan(64), torch.arange(4, dtype=torch.int32, device="cuda")
    norm = binding.HeadNorm(torch.ones(64, device="cuda"))
    x = torch.ones(4, 2, 64, device="cuda")
    for bad in (lambda: binding.HeadNorm(torch.ones(64)), lambda: binding.HeadNorm(torch.ones(64, device="cuda").half()),
                lambda: binding.HeadNorm(torch.ones(2, 64, device="cuda")),
                lambda: binding.norm_rope(plan, binding.HeadNorm(torch.ones(32, device="cuda")), pos, x),
                lambda: binding.norm_rope(plan, norm, pos[:3], x), lambda: binding.norm_rope(plan, norm, pos, x.half()),
                lambda: binding.norm_rope(plan, norm, pos, x[:, :, :32]), lambda: binding.norm_rope(plan, norm, pos, x[0]),
                lambda: binding.norm_rope(plan, binding.HeadNorm(torch.ones(64, device="cuda"), eps=math.nan), pos, x),
                lambda: binding.norm_rope(plan, binding.HeadNorm(torch.ones(64, device="cuda"), offset=math.inf), pos, x),
                lambda: binding.norm_rope_grad(plan, norm, pos, x, x.to(torch.bfloat16)),
                lambda: binding.norm_rope_grad(plan, norm, pos, x, x[:3]),
                lambda: binding.norm_rope_grad(plan, norm, pos, x, x, dw=torch.empty(32, device="cuda")),
                lambda: binding.norm_rope_grad(plan, norm, torch.arange(4096, dtype=torch.int32, device="cuda"),
                                               x[:1].expand(4096, 2, 64).contiguous(), x[:1].expand(4096, 2, 64).contiguous(),
                                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(binding.GdnSpecError):
            bad()
