"""Attention of packed prompts over the paged cache against the 64-bit definition (bounds: prompt_case.py)."""
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests.prompt_case import FP32_NOISE, HALF_ULP, Prompts
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu

EDGE = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300]


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_counts_around_tiles_and_pages(io, D, G):
    """Prompts of every length around the tiles, without and behind contexts that end anywhere."""
    Prompts(1, io, 2 * G, 2, D, 16, counts=EDGE, lens=[0] * len(EDGE)).check()
    Prompts(2, io, 2 * G, 2, D, 16, counts=EDGE, lens=EDGE[::-1]).check()


@pytest.mark.parametrize("io,HQ,HKV,D,P", [
    ("bf16", 2, 2, 64, 16), ("bf16", 16, 2, 256, 64), ("bf16", 32, 8, 128, 32), ("bf16", 7, 1, 128, 128),
    ("bf16", 16, 2, 256, 256), ("bf16", 4, 2, 64, 64), ("bf16", 16, 2, 64, 128), ("bf16", 8, 1, 256, 16),
    ("bf16", 48, 1, 128, 64), ("bf16", 20, 4, 96, 16), ("bf16", 6, 3, 40, 32), ("bf16", 5, 1, 192, 128),
    ("bf16", 6, 2, 200, 64), ("bf16", 64, 1, 8, 256), ("bf16", 127, 1, 64, 32), ("bf16", 128, 1, 128, 128),
    ("bf16", 130, 1, 128, 32), ("bf16", 300, 1, 64, 16), ("bf16", 129, 1, 256, 64),
    ("fp32", 2, 2, 64, 16), ("fp32", 8, 1, 256, 32), ("fp32", 16, 4, 128, 64), ("fp32", 9, 3, 8, 16),
    ("fp32", 5, 1, 200, 256), ("fp32", 65, 1, 64, 32), ("fp32", 140, 1, 24, 16)])
def test_types_heads_and_pages(io, HQ, HKV, D, P):
    c = Prompts(3, io, HQ, HKV, D, P, counts=[70, 1, 5, 300, 33], lens=[0, 411, 98, 130, 64])
    c.check()
    assert binding.prompt_attn_path(c.cache, HQ) == ("tc" if io == "bf16" else "generic")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_empty_rows_padding_and_tokens_of_no_row(io, D):
    """Rows of no token, a padding row in the middle and at both ends, tokens before the first row and behind
    the last, which are left as they were."""
    c = Prompts(4, io, 4, 2, D, 32, counts=[9, 0, 130, 40, 0, 1, 65], lens=[0, 70, 33, 0, 129, 500, 7],
                slots=[-1, 1, 2, -1, 4, 5, -1], lead=3, tail=50)
    out, lse = c.check()
    assert (out[3:12] == 0).all() and torch.isneginf(lse[142:182]).all()
    c = Prompts(5, io, 4, 2, D, 32, counts=[0, 0], lens=[0, 70], tail=4)
    c.check()


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("HQ,HKV,D,P", [(4, 2, 128, 16), (2, 2, 64, 64), (8, 1, 256, 128), (1, 1, 128, 128), (6, 2, 96, 32)])
def test_later_tokens_may_hold_anything(io, HQ, HKV, D, P):
    """A token with a NaN key and NaN or infinite values changes only itself and those behind it; several a tile, some in
    the tile before the last, in rows that start inside a tile."""
    counts, lens = [61, 200, 300, 7], [0, 100, 33, 250]
    c, clean = (Prompts(6, io, HQ, HKV, D, P, counts, lens) for _ in range(2))
    bads = {0: [5, 60], 1: [17, 18, 150], 2: [130, 299], 3: [3]}
    for s, at in bads.items():
        for n, i in enumerate(at):
            page, off = c.row(s, int(c.lens[s]) + i)
            if n % 2 == 0:
                c.k[0, page, 0, off] = math.nan
            c.v[0, page, 0, off, :] = math.inf if s % 2 else math.nan
    got, want = c.call()[0].float().cpu().numpy(), clean.call()[0].float().cpu().numpy()
    G = HQ // HKV
    for s, at in bads.items():
        a, e = c.starts[s], c.starts[s + 1]
        first = a + min(at)
        assert np.array_equal(got[a:first], want[a:first])           # before the first of them: the same bits
        assert not np.isfinite(got[first:e, :G]).any()
        assert np.array_equal(got[a:e, G:], want[a:e, G:])            # the other kv head's


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("HQ,HKV,D", [(4, 2, 128), (8, 2, 64), (4, 1, 256)])
def test_infinite_values_reach_the_tokens_that_see_them(io, HQ, HKV, D):
    """Only the values of some tokens are infinite in some dims: they and those behind them are infinite there and as ever
    elsewhere."""
    c = Prompts(7, io, HQ, HKV, D, 64, counts=[150, 300], lens=[61, 200])
    dims = torch.arange(0, D, 3)
    for s, at in ((0, [100]), (1, [7, 290])):
        for i in at:
            page, off = c.row(s, int(c.lens[s]) + i)
            c.v[0, page, :, off, dims] = math.inf
    got = c.call()[0].double().cpu().numpy()
    want, _, spread = c.expect()
    fin = np.isfinite(want)
    assert fin.any() and (~fin).any()
    # a masked infinity is 0 times infinity in the definition's product: what it gives NaN for is seen token by token
    seen = np.zeros_like(fin)
    for s, at in ((0, [100]), (1, [7, 290])):
        seen[c.starts[s] + min(at):c.starts[s + 1], :, ::3] = True
    assert np.array_equal(np.isposinf(got), seen)
    c.v = torch.where(torch.isfinite(c.v), c.v, torch.zeros_like(c.v))
    want, _, spread = c.expect()
    err = np.where(seen, 0, np.abs(np.where(seen, 0, got) - want))
    assert (err <= c.bound(want, spread)).all()


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [128, 256])
def test_mixed_with_decode_rows_split_and_joined(io, D):
    """Single tokens behind long, uneven contexts beside prompts: items cut over many blocks; twice the same."""
    c = Prompts(8, io, 4, 1, D, 128, counts=[1, 300, 1, 1, 2, 64], lens=[20011, 0, 7000, 129, 3000, 5000], poison=False)
    a, la = c.check()
    b, lb = c.call()
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("io,HQ,HKV,D,n", [("bf16", 4, 1, 128, 5000), ("bf16", 2, 2, 64, 3333), ("bf16", 8, 1, 256, 2500),
                                           ("fp32", 2, 1, 128, 2100)])
def test_one_long_prompt(io, HQ, HKV, D, n):
    Prompts(9, io, HQ, HKV, D, 64, counts=[n], lens=[77], poison=False).check()


@pytest.mark.parametrize("HQ,HKV,D,counts,lens", [(8, 8, 256, [300, 1, 290], [13000, 5000, 12000]),
                                                  (32, 16, 128, [290, 300], [26000, 13000])])
def test_contexts_larger_than_a_wave(HQ, HKV, D, counts, lens):
    """Rows of several blocks whose keys and values are more than are gone through at a time (96 MB)."""
    assert (lens[0] + lens[-1]) * HKV * D * 4 > 96 << 20
    Prompts(21, "bf16", HQ, HKV, D, 64, counts=counts, lens=lens, poison=False).check()


def test_more_rows_than_a_block_scans_and_layers():
    """700 rows of 0 to 6 tokens, the last of three layers."""
    r = np.random.default_rng(10)
    Prompts(10, "bf16", 4, 2, 64, 16, counts=r.integers(0, 7, 700), lens=r.integers(0, 90, 700), layers=3, layer=2,
            lead=2, tail=5).check()
    Prompts(11, "fp32", 4, 2, 64, 16, counts=r.integers(0, 7, 700), lens=r.integers(0, 90, 700), layers=3, layer=2).check()


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_scale(io):
    """From almost uniform weights to a single one.  Large scores carry a larger absolute error, 2^-22 of their size, so the
    last case compares where one weight is all there is."""
    Prompts(12, io, 4, 2, 128, 32, counts=[150, 65], lens=[100, 65], scale=1e-3).check()
    c = Prompts(12, io, 4, 2, 128, 32, counts=[150, 65], lens=[100, 65], scale=30.0)
    out, _ = c.call()
    want, _, _ = c.expect()
    assert np.max(np.abs(out.double().cpu().numpy() - want)) <= 2e-2


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_maximum_that_climbs(D):
    """Keys that grow along the row, so that the running maximum moves in almost every tile: scores rise by some 20 in
    powers of two a tile, over 30 tiles.  Scores up to 300 carry an error of 2^-24 times the root of D times their size,
    some 3e-4, by which every probability may be off."""
    c = Prompts(13, "bf16", 2, 1, D, 64, counts=[3, 200], lens=[4000, 3800], poison=False)
    c.q = torch.ones_like(c.q)
    for s in range(2):
        for i in range(int(c.lens[s] + c.counts[s])):
            page, off = c.row(s, i)
            c.k[0, page, 0, off] = (0.05 + 0.0005 * i) * 16 / D ** 0.5
    c.scale = D ** -0.5 * D ** 0.5 / 4
    out, lse = c.call()
    want, wl, spread = c.expect()
    assert (np.abs(out.double().cpu().numpy() - want) <= c.bound(want, spread) + 1e-3 * spread).all()
    assert np.max(np.abs(lse.double().cpu().numpy() - wl)) <= 1e-3


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_another_stream_and_a_graph(io):
    c = Prompts(14, io, 8, 2, 128, 64, counts=[100, 300, 1], lens=[500, 0, 3000])
    want, wl = c.check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gl = c.call()
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(gl, wl)
    given, _ = c.call(stream=s)
    s.synchronize()
    cache, slots, starts, q = c.cache, torch.from_numpy(c.slots).cuda(), torch.from_numpy(c.starts).cuda(), c.q.cuda()
    work = torch.empty(binding.prompt_attn_workspace(cache, 3, c.N, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.prompt_attn(cache, 0, slots, starts, q, scale=c.scale, out=out, workspace=work)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # the captured call follows the counts on the device: the second row is empty, most tokens are nobody's (the work
    # is cut elsewhere then, so the first row's bits may differ)
    c.starts = np.array([0, 100, 100, 101], np.int32)
    starts.copy_(torch.from_numpy(c.starts))
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    want, _, spread = c.expect()
    assert (out[101:] == 7).all()
    assert (np.abs(out[:101].double().cpu().numpy() - want[:101]) <= c.bound(want, spread)[:101]).all()


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_a_workspace_does_for_fewer_rows_and_tokens(io):
    """One that was made for 64 rows and 1200 tokens takes one row of 1100 (its part of the line may be cut finer), and
    the gradient's every smaller count."""
    c = Prompts(30, io, 2, 2, 64, 64, counts=[1100], lens=[40])
    cache = c.upload()
    large = binding.KvCache(1, 8192, 2, 64, 64, 1, 4, io)                # more pages than L2 holds
    for kv in (cache, large):
        most = binding.prompt_attn_workspace(kv, 64, 1200, 2)
        for B, N in ((1, 0), (1, 1), (1, 1100), (1, 1200), (2, 700), (63, 1199), (64, 64), (0, 0)):
            assert binding.prompt_attn_workspace(kv, B, N, 2) <= most, (B, N)
    slots, starts = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    binding.prompt_attn(large, 0, slots, starts, c.q.cuda(),
                        workspace=torch.empty(binding.prompt_attn_workspace(large, 64, 1200, 2), dtype=torch.uint8, device="cuda"))
    c.check(workspace=torch.empty(binding.prompt_attn_workspace(cache, 64, 1200, 2), dtype=torch.uint8, device="cuda"))
    before = 0
    for n in (0, 1, 2, 100, 303, 304, 305, 1023, 1024, 1025, 2047, 2048, 4096, 8192, 16384, 100000):
        now = binding.norm_rope_grad_workspace(n, 4, 128)
        assert now >= before, n
        before = now


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_refused_rows_report_and_give_zeros(io):
    c = Prompts(15, io, 4, 2, 128, 32, counts=[4, 4, 5, 70, 4], lens=[40, 50, 60, 70], slots=[0, 9, 1, 2, 3])
    cache = c.upload()
    cache.length[2] = -1
    cache.n_pages[3] = 2                                  # 70 tokens do not fit in two pages
    out, lse = c.call()
    assert binding.kv_read_status(cache) == binding.ST_SLOT_OOR | binding.ST_CURSOR_CORRUPT
    s = c.starts
    for b in (1, 3, 4):
        assert (out[s[b]:s[b + 1]] == 0).all() and torch.isneginf(lse[s[b]:s[b + 1]]).all()
    assert (out[:4] != 0).any() and (out[s[2]:s[3]] != 0).any()
    cache.length[2] = 70
    cache.n_pages[3] = 3
    cache.length[3] = 94                                  # 94 fit, 98 do not
    c.call()
    assert binding.kv_read_status(cache) == binding.ST_SLOT_OOR | binding.ST_NO_PAGES
    cache.length[3] = 70
    cache.page_table[3, 1] = c.num_pages + 5
    c.call()
    assert binding.kv_read_status(cache) == binding.ST_SLOT_OOR | binding.ST_PAGE_OOR


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_starts_that_do_not_ascend_or_leave_the_tensors(io):
    """A row whose two entries are no range owns nothing and is reported; the others are as ever."""
    c = Prompts(16, io, 4, 2, 64, 32, counts=[20, 30, 40], lens=[10, 0, 70])
    c.check()
    want, _, spread = c.expect()
    cache = c.cache
    good = c.starts.copy()
    for bad, row in (([0, 20, 50, c.N + 1], 2), ([-3, 20, 50, 90], 0), ([0, 20, 50, 45], 2)):
        c.starts = np.array(bad, np.int32)
        out, lse = c.call()
        assert binding.kv_read_status(cache) == binding.ST_ACCEPT_RANGE
        mine = slice(good[row], good[row + 1])
        assert (out[mine] == 7).all() and (lse[mine] == 7).all()
        rest = np.ones(c.N, bool)
        rest[mine] = False
        assert (np.abs(out.double().cpu().numpy() - want) <= c.bound(want, spread))[rest].all()


def test_binding_refuses():
    c = Prompts(17, "bf16", 4, 2, 128, 32, counts=[9], lens=[40])
    cache, q, s = c.upload(), c.q.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    st = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    assert binding.prompt_attn(cache, 0, s, st, q).shape == q.shape
    assert binding.prompt_attn(cache, 0, s[:0], st[:1], q).shape == q.shape
    assert binding.prompt_attn(cache, 0, s, st, q[:0]).shape == (0, 4, 128)
    for bad in (lambda: binding.prompt_attn(cache, 1, s, st, q), lambda: binding.prompt_attn(cache, 0, s, st, q.float()),
                lambda: binding.prompt_attn(cache, 0, s, st, q[:, :3]), lambda: binding.prompt_attn(cache, 0, s, st[:1], q),
                lambda: binding.prompt_attn(cache, 0, s, st, q[None]), lambda: binding.prompt_attn(cache, 0, s, st.long(), q),
                lambda: binding.prompt_attn(cache, 0, s, st, q, scale=0.0),
                lambda: binding.prompt_attn(cache, 0, s, st, q, scale=math.nan),
                lambda: binding.prompt_attn(cache, 0, s, st, q, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                lambda: binding.prompt_attn(cache, 0, s, st, q.cpu()), lambda: binding.prompt_attn(cache, 0, s.cpu(), st, q)):
        with pytest.raises(binding.GdnSpecError):
            bad()


@pytest.mark.parametrize("HQ,HKV,D", [(8, 2, 128), (8, 2, 256), (4, 1, 64)])
def test_a_wait_that_runs_out_is_reported(HQ, HKV, D):
    """With the wait limit at zero the first wait on copied data gives up: the copies in flight are drained, the call
    returns with TIMEOUT, and the next call is right."""
    c = Prompts(18, "bf16", HQ, HKV, D, 32, counts=[300, 1, 90], lens=[700, 90, 0])
    cache = c.upload()
    prev = binding.set_wait_limit(0)
    try:
        c.call()
        st = binding.kv_read_status(cache)
    finally:
        binding.set_wait_limit(binding.WAIT_LIMIT_DEFAULT)
    assert prev == 1 << 20 and st == binding.ST_TIMEOUT
    c.check()


def test_the_same_call_gives_the_same_bits():
    """Forty calls of each layout, other work between them."""
    other = torch.zeros(1 << 22, device="cuda")
    for io, HQ, HKV, D in (("bf16", 8, 2, 128), ("bf16", 2, 1, 64), ("bf16", 8, 1, 256), ("fp32", 4, 1, 128)):
        c = Prompts(19, io, HQ, HKV, D, 64, counts=[700, 1, 65, 300], lens=[0, 3000, 900, 64])
        a, la = c.call()
        for _ in range(40):
            other.add_(1.0)
            b, lb = c.call()
            assert torch.equal(a, b) and torch.equal(la, lb)
        assert binding.kv_read_status(c.cache) == 0


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_a_pool_past_32_bits(io):
    """Pages whose elements and bytes lie past 2^31 and 2^32: the same bits as from a small pool."""
    HQ, HKV, D, P = 4, 2, 256, 256
    c = Prompts(20, io, HQ, HKV, D, P, counts=[90, 300, 1], lens=[700, 3, 256], layers=2, layer=1, poison=False)
    want, wl = c.call()
    big_pages = 10000                                        # 2 layers of 10000 pages: 2.6e9 elements
    to = np.linspace(0, big_pages - 1, c.num_pages).astype(np.int32)[::-1].copy()
    table = np.where(c.table >= 0, to[np.maximum(c.table, 0)], -1).astype(np.int32)
    where = torch.from_numpy(to).long().cuda()
    pool = [torch.empty(2, big_pages, HKV, P, D, dtype=ref.TORCH[io], device="cuda") for _ in range(2)]
    for x, y in zip(pool, (c.cache.k, c.cache.v)):
        x[:, where] = y
    c.cache = binding.KvCache(2, big_pages, HKV, P, D, len(c.lens), table.shape[1], io, tensors={
        "k": pool[0], "v": pool[1], "page_table": torch.from_numpy(table).cuda(),
        "n_pages": torch.from_numpy(c.n_pages).cuda(), "length": torch.from_numpy(c.lens).cuda()})
    got, gl = c.call()
    assert binding.kv_read_status(c.cache) == 0 and torch.equal(got, want) and torch.equal(gl, wl)
