"""Attention of drafted windows over the paged cache against the 64-bit definition.

Bounds, per output element, from how it is computed: the result is rounded once to the
I/O type (half a unit: at most 2^-8 of it in bf16, 2^-24 in fp32); with bf16 the
probabilities are rounded before the second product, each by at most 2^-8 of itself, so by at
most 2^-8 of sum p |v| in all; scores are fp32 sums of D products, whose error (some 2^-24 times
the root of D times their size) moves every probability by a few 1e-6 of itself: 2e-5
of sum p |v| is allowed for it and for the sums.  lse likewise: 2e-5 absolute (scores
here are below 16, times the same relative error).
"""
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu

HALF_ULP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
FP32_NOISE = 2e-5


class Case:
    """A layer of a cache with scattered pages, every unused row of the pool poisoned."""

    def __init__(self, seed, io, T, HQ, HKV, D, P, lens, slots=None, layers=1, layer=0, poison=True,
                 counts=None, tree="tree", scale=None):
        r = self.rng = np.random.default_rng(seed)
        self.io, self.T, self.HQ, self.D, self.P, self.layer = io, T, HQ, D, P, layer
        self.lens = np.asarray(lens, np.int32)
        self.slots = np.asarray(range(len(lens)) if slots is None else slots, np.int32)
        B = len(self.slots)
        self.counts = np.full(B, T, np.int32) if counts is None else np.asarray(counts, np.int32)
        self.scale = D ** -0.5 if scale is None else scale
        need = int(sum(-(-(int(n) + T) // P) for n in lens))
        self.num_pages, max_pages = need + 2, max(-(-(int(n) + T) // P) for n in lens) + 1
        self.table, self.n_pages = ref.pages_for(r, self.lens, T, P, self.num_pages, max_pages)
        shape = (layers, self.num_pages, HKV, P, D)
        self.k, self.v = ref.draw(r, shape, io), ref.draw(r, shape, io)
        if poison:   # what no token of the window or before it owns may be anything
            live = np.zeros((self.num_pages, P), bool)
            for b, s in enumerate(self.slots):
                if 0 <= s < len(self.lens):
                    i = np.arange(int(self.lens[s]) + int(self.counts[b]))
                    live[self.table[s, i // P], i % P] = True
            dead = torch.from_numpy(~live)[None, :, None, :, None].expand(shape)
            for x, bad in ((self.k, math.nan), (self.v, math.inf)):
                x.masked_fill_(dead, bad)
        self.q = ref.draw(r, (B, T, HQ, D), io)
        if tree == "chain":
            self.masks = [[(1 << (t + 1)) - 1 for t in range(T)] for _ in range(B)]
        else:
            self.masks = [[int(m) for m in ref.ancestors(ref.random_tree(r, T))] for _ in range(B)]
        self.tree = tree
        self.cache = None

    def upload(self):
        t = {"k": self.k.cuda(), "v": self.v.cuda(), "page_table": torch.from_numpy(self.table).cuda(),
             "n_pages": torch.from_numpy(self.n_pages).cuda(), "length": torch.from_numpy(self.lens).cuda()}
        L, NP, HKV, P, D = self.k.shape
        self.cache = binding.KvCache(L, NP, HKV, P, D, len(self.lens), self.table.shape[1], self.io, tensors=t)
        return self.cache

    def call(self, **kw):
        cache = self.cache or self.upload()
        B = len(self.slots)
        mask = None
        if self.tree != "chain":
            mask = torch.from_numpy(np.array(self.masks, np.uint64).view(np.int64)).cuda()
        ragged = (self.counts != self.T).any()
        out = torch.full((B, self.T, self.HQ, self.D), 7.0, dtype=ref.TORCH[self.io], device="cuda")
        lse = torch.full((B, self.T, self.HQ), 7.0, device="cuda")
        binding.tree_attn(cache, self.layer, torch.from_numpy(self.slots).cuda(), self.q.cuda(), mask,
                          torch.from_numpy(self.counts).cuda() if ragged else None, scale=self.scale, out=out,
                          lse=lse, **kw)
        return out, lse

    def expect(self):
        f = lambda x: x.double().numpy()  # noqa: E731
        return ref.attention(f(self.q), f(self.k[self.layer]), f(self.v[self.layer]), self.table, self.slots,
                             self.lens, self.masks, self.counts, self.scale)

    def check(self, **kw):
        out, lse = self.call(**kw)
        assert binding.kv_read_status(self.cache) == 0
        want, want_lse, spread = self.expect()
        got = out.double().cpu().numpy()
        p_round = HALF_ULP["bf16"] if self.io == "bf16" else 0.0
        bound = HALF_ULP[self.io] * np.abs(want) + (p_round + FP32_NOISE) * spread * (1 + 2.0 ** -8)
        assert np.isfinite(got).all()
        worst = np.max(np.abs(got - want) - bound)
        assert worst <= 0, (worst, np.max(np.abs(got - want)))
        gl = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(gl), np.isneginf(want_lse))
        fin = np.isfinite(want_lse)
        assert np.max(np.abs(gl[fin] - want_lse[fin]), initial=0.0) <= 2e-5
        return out, lse


EDGE = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 300]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths_around_tiles_and_pages(io, D):
    Case(1, io, T=5, HQ=6, HKV=2, D=D, P=16, lens=EDGE).check()


@pytest.mark.parametrize("io,T,HQ,HKV,D,P", [
    ("bf16", 1, 2, 2, 64, 16), ("bf16", 1, 16, 2, 256, 64), ("bf16", 1, 32, 8, 128, 32),
    ("bf16", 2, 7, 1, 128, 128), ("bf16", 8, 16, 2, 256, 256), ("bf16", 33, 4, 2, 64, 64),
    ("bf16", 64, 2, 1, 128, 16), ("bf16", 64, 16, 2, 64, 32), ("bf16", 64, 16, 2, 128, 128),
    ("bf16", 64, 8, 1, 256, 64), ("bf16", 3, 48, 1, 128, 64), ("bf16", 7, 20, 4, 96, 16),
    ("bf16", 5, 6, 3, 40, 32), ("bf16", 40, 9, 3, 128, 64),
    ("fp32", 1, 2, 2, 64, 16), ("fp32", 1, 8, 1, 256, 32), ("fp32", 8, 16, 4, 128, 64),
    ("fp32", 64, 8, 2, 64, 128), ("fp32", 3, 9, 3, 8, 16), ("fp32", 6, 5, 1, 200, 256)])
@pytest.mark.parametrize("tree", ["chain", "tree"])
def test_types_heads_windows_pages(io, T, HQ, HKV, D, P, tree):
    Case(2, io, T, HQ, HKV, D, P, lens=[211, 0, 98, 640], tree=tree).check()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_rows_without_anything_and_padding(io):
    """Counts from 0 to T, a padding row, an empty context, nodes whose mask is empty."""
    c = Case(3, io, T=6, HQ=4, HKV=2, D=128, P=32, lens=[0, 70, 33, 0, 129], slots=[0, 1, -1, 2, 3, 4],
             counts=[6, 0, 3, 2, 1, 5])
    c.masks[0] = [0, 0b10, 0, 0b1011, 0, 0b100000]      # slot 0 has no context: rows 0, 2, 4 see nothing
    c.masks[5] = [0, 1, 0, 7, 0, 0]                      # slot 4 has one: they see the context alone
    out, lse = c.check()
    o = out.float().cpu().numpy()
    assert (o[0, 0] == 0).all() and (o[1] == 0).all() and (o[2] == 0).all() and (o[4, 1:] == 0).all()
    assert np.isneginf(lse.cpu().numpy()[2]).all()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T,HQ,HKV,D", [(8, 4, 2, 128), (64, 8, 2, 128), (8, 4, 1, 256), (5, 3, 3, 64)])
def test_masked_drafts_may_hold_anything(io, T, HQ, HKV, D):
    """A draft with NaN keys and NaN or infinite values changes only the nodes below it."""
    lens = [61, 128, 0, 250]
    c = Case(4, io, T, HQ, HKV, D, 16, lens=lens)
    clean = Case(4, io, T, HQ, HKV, D, 16, lens=lens)
    bad = 2
    sees = np.array([[m >> bad & 1 for m in row] for row in c.masks], bool)
    for b, s in enumerate(c.slots):
        i = int(c.lens[s]) + bad
        page, off = int(c.table[s, i // 16]), i % 16
        c.k[0, page, 0, off] = math.nan
        c.v[0, page, 0, off, :] = math.inf if b % 2 else math.nan
    got, lse = c.call()
    want, wl = clean.call()
    G = HQ // HKV
    g, w = got.float().cpu().numpy(), want.float().cpu().numpy()
    for b in range(len(lens)):
        for t in range(T):
            mine = slice(0, G)                           # the heads of kv head 0
            if sees[b, t]:
                assert np.isnan(g[b, t, mine]).all()
            else:
                assert np.array_equal(g[b, t, mine], w[b, t, mine])
            assert np.array_equal(g[b, t, G:], w[b, t, G:])


@pytest.mark.parametrize("T,HQ,HKV,D", [(8, 4, 2, 128), (64, 8, 2, 128), (8, 4, 1, 256)])
def test_infinite_values_reach_the_nodes_that_see_them(T, HQ, HKV, D):
    """Only the values of one draft are infinite in some dims: nodes below it are infinite
    there and as ever elsewhere."""
    c = Case(5, "bf16", T, HQ, HKV, D, 64, lens=[61, 200])
    dims = torch.arange(0, D, 3)
    for s in (0, 1):
        i = int(c.lens[s]) + 1
        c.v[0, int(c.table[s, i // 64]), :, i % 64, dims] = math.inf
    out, _ = c.call()
    want, _, spread = c.expect()
    got = out.double().cpu().numpy()
    fin = np.isfinite(want)
    assert fin.any() and (~fin).any()
    assert np.array_equal(np.isposinf(got), np.isposinf(want))
    sp = np.where(np.isfinite(spread), spread, 0)
    err = np.abs(np.where(fin, got, 0) - np.where(fin, want, 0))
    assert (err <= 2.0 ** -8 * np.abs(np.where(fin, want, 0)) + (2.0 ** -8 + FP32_NOISE) * sp * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_long_contexts_are_split_and_joined(io):
    """Few rows with long, uneven contexts: items cut over many blocks; twice the same."""
    c = Case(6, io, T=3, HQ=4, HKV=1, D=128, P=128, lens=[20011, 1, 7000, 129], poison=False)
    a, la = c.check()
    b, lb = c.call()
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_many_rows_share_pages_and_layers():
    """More rows than a block scans at once, slots that repeat pages, the last of three layers.  Rows that
    are alike may be cut at different places, so they agree within the bounds."""
    lens = [40, 90, 3, 64, 17]
    c = Case(7, "bf16", T=2, HQ=4, HKV=2, D=64, P=16, lens=lens, slots=[i % 5 for i in range(700)], layers=3, layer=2)
    c.q = c.q[:5].repeat(140, 1, 1, 1)
    c.masks = [c.masks[i % 5] for i in range(700)]
    out, lse = c.call()
    assert binding.kv_read_status(c.cache) == 0
    c.q, c.masks, c.slots, c.counts = c.q[:5], c.masks[:5], c.slots[:5], c.counts[:5]
    want, want_lse, spread = (x[None] for x in c.expect())
    got = out.double().cpu().numpy().reshape(140, 5, 2, 4, 64)
    bound = HALF_ULP["bf16"] * np.abs(want) + (HALF_ULP["bf16"] + FP32_NOISE) * spread * (1 + 2.0 ** -8)
    assert (np.abs(got - want) <= bound).all()
    assert np.max(np.abs(lse.double().cpu().numpy().reshape(140, 5, 2, 4) - want_lse)) <= 2e-5
    small, _ = c.call()
    assert small.shape == (5, 2, 4, 64)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
def test_scale(scale):
    """From almost uniform weights to a single one.  Large scores carry a larger absolute error,
    2^-22 of their size, so the last case compares where one weight is all there is."""
    c = Case(8, "bf16", T=4, HQ=4, HKV=2, D=128, P=32, lens=[300, 65], scale=scale)
    if scale < 2:
        if scale == 1.0:
            c.q = (c.q.float() / 4).to(torch.bfloat16)
        c.check()
        return
    out, _ = c.call()
    want, _, _ = c.expect()
    assert np.max(np.abs(out.double().cpu().numpy() - want)) <= 2e-2


def test_another_stream_and_a_graph():
    c = Case(9, "bf16", T=4, HQ=8, HKV=2, D=128, P=64, lens=[500, 3000])
    want, wl = c.check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gl = c.call()
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(gl, wl)
    cache, slots, q = c.cache, torch.from_numpy(c.slots).cuda(), c.q.cuda()
    mask = torch.from_numpy(np.array(c.masks, np.uint64).view(np.int64)).cuda()
    work = torch.empty(binding.tree_attn_workspace(cache, 2, 4, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.tree_attn(cache, 0, slots, q, mask, scale=c.scale, out=out, workspace=work)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_refused_rows_report_and_give_zeros():
    c = Case(10, "bf16", T=4, HQ=4, HKV=2, D=128, P=32, lens=[40, 50, 60, 70], slots=[0, 9, 1, 2, 3])
    c.counts[:] = [4, 4, 5, 4, 4]
    cache = c.upload()
    cache.length[2] = -1
    cache.n_pages[3] = 2                                 # 70 tokens do not fit in two pages
    out, lse = c.call()
    st = binding.kv_read_status(cache)
    assert st == binding.ST_SLOT_OOR | binding.ST_ACCEPT_RANGE | binding.ST_CURSOR_CORRUPT
    assert (out[1:] == 0).all() and torch.isneginf(lse[1:]).all()
    c.counts[:] = 4
    cache.length[2] = 60
    cache.n_pages[3] = 3                                 # 70 fit, 74 do too; 100 do not
    cache.length[3] = 94
    out, _ = c.call()
    assert binding.kv_read_status(cache) == binding.ST_SLOT_OOR | binding.ST_NO_PAGES
    assert (out[1] == 0).all() and (out[4] == 0).all() and (out[2:4] != 0).any()
    cache.length[3] = 70
    cache.page_table[3, 1] = c.num_pages + 5
    c.call()
    assert binding.kv_read_status(cache) == binding.ST_SLOT_OOR | binding.ST_PAGE_OOR


def test_binding_refuses():
    c = Case(11, "bf16", T=4, HQ=4, HKV=2, D=128, P=32, lens=[40])
    cache, q, s = c.upload(), c.q.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    ok = binding.tree_attn(cache, 0, s, q)
    assert ok.shape == q.shape
    for bad in (lambda: binding.tree_attn(cache, 1, s, q), lambda: binding.tree_attn(cache, 0, s, q.float()),
                lambda: binding.tree_attn(cache, 0, s, q[:, :, :3]), lambda: binding.tree_attn(cache, 0, s, q[0]),
                lambda: binding.tree_attn(cache, 0, s, q.transpose(1, 2)),
                lambda: binding.tree_attn(cache, 0, s, q, scale=0.0),
                lambda: binding.tree_attn(cache, 0, s, q, scale=math.nan),
                lambda: binding.tree_attn(cache, 0, s, q, tree_mask=torch.zeros(1, 4, device="cuda")),
                lambda: binding.tree_attn(cache, 0, s, q, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                lambda: binding.tree_attn(cache, 0, s, q.repeat(1, 17, 1, 1)),
                lambda: binding.tree_attn(cache, 0, s.cpu(), q)):
        with pytest.raises(binding.GdnSpecError):
            bad()


@pytest.mark.parametrize("T,HQ,HKV,D,lens", [(4, 8, 2, 128, [700, 90]), (64, 8, 2, 128, [700, 90]),
                                             (4, 8, 2, 256, [700, 90]), (33, 8, 1, 64, [5, 3000, 0])])
def test_a_wait_that_runs_out_is_reported(T, HQ, HKV, D, lens):
    """With the wait limit at zero the first wait on copied data gives up: the copies in flight
    are drained, the call returns with TIMEOUT, and the next call is right."""
    c = Case(12, "bf16", T=T, HQ=HQ, HKV=HKV, D=D, P=32, lens=lens)
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
    """Forty calls of each layout of streams, other work between them."""
    other = torch.zeros(1 << 22, device="cuda")
    for T, HQ, HKV, D, lens in ((2, 8, 2, 128, [3000, 17, 900, 64]), (64, 16, 2, 128, [1500, 130]),
                                (7, 8, 1, 256, [2000, 333, 1]), (40, 8, 2, 64, [800, 65])):
        c = Case(13, "bf16", T=T, HQ=HQ, HKV=HKV, D=D, P=64, lens=lens)
        a, la = c.call()
        for _ in range(40):
            other.add_(1.0)
            b, lb = c.call()
            assert torch.equal(a, b) and torch.equal(la, lb)
        assert binding.kv_read_status(c.cache) == 0


@pytest.mark.parametrize("io,T,HQ,HKV,D,P", [
    ("fp32", 1, 4, 1, 128, 64), ("fp32", 2, 4, 2, 256, 16), ("fp32", 4, 1, 1, 136, 32),      # 4 rows a tile
    ("fp32", 2, 8, 2, 64, 16), ("fp32", 7, 2, 2, 128, 128),                                  # 8
    ("fp32", 3, 8, 2, 128, 16), ("fp32", 6, 4, 2, 256, 64), ("fp32", 11, 1, 1, 64, 32),      # 12
    ("fp32", 16, 2, 2, 200, 64), ("fp32", 3, 10, 2, 64, 16),                                 # 16
    ("fp32", 6, 4, 1, 64, 16), ("fp32", 8, 3, 1, 256, 64), ("fp32", 5, 18, 2, 128, 32),      # 24, once and twice
    ("fp32", 9, 8, 2, 256, 32), ("fp32", 64, 3, 1, 128, 256), ("fp32", 17, 2, 1, 24, 16),    # 32, several tiles
    ("bf16", 2, 130, 1, 128, 32), ("bf16", 1, 300, 2, 64, 16), ("bf16", 3, 129, 1, 256, 64)])
def test_the_cuda_core_kernel(io, T, HQ, HKV, D, P):
    """Every size of its query tiles, and bf16 with more than 128 heads a kv head."""
    c = Case(14, io, T, HQ, HKV, D, P, lens=[33, 0, 500, 31, 7])
    c.check()
    assert binding.tree_attn_path(c.cache, T, HQ) == "generic"


@pytest.mark.parametrize("T,HQ,HKV,D", [(8, 4, 2, 128), (2, 2, 1, 64), (40, 8, 2, 256), (3, 4, 1, 72)])
def test_infinite_values_in_fp32(T, HQ, HKV, D):
    """As with bf16: a draft's infinite values reach the nodes below it, in their dims, and no other."""
    c = Case(15, "fp32", T=T, HQ=HQ, HKV=HKV, D=D, P=64, lens=[61, 200, 30])
    dims = torch.arange(0, D, 3)
    for s in range(3):
        i = int(c.lens[s]) + 1
        c.v[0, int(c.table[s, i // 64]), :, i % 64, dims] = math.inf
    out, _ = c.call()
    want, _, spread = c.expect()
    got = out.double().cpu().numpy()
    fin = np.isfinite(want)
    assert fin.any() and (~fin).any()
    assert np.array_equal(np.isposinf(got), np.isposinf(want))
    sp = np.where(np.isfinite(spread), spread, 0)
    err = np.abs(np.where(fin, got, 0) - np.where(fin, want, 0))
    assert (err <= 2.0 ** -24 * np.abs(np.where(fin, want, 0)) + FP32_NOISE * sp).all()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_a_pool_past_32_bits(io):
    """Pages whose elements and bytes lie past 2^31 and 2^32: the same bits as from a small pool."""
    T, HQ, HKV, D, P = 5, 4, 2, 256, 256
    c = Case(16, io, T, HQ, HKV, D, P, lens=[700, 3, 256], layers=2, layer=1, poison=False)
    want, wl = c.call()
    small, big_pages = c.cache, 10000                        # 2 layers of 10000 pages: 2.6e9 elements
    to = np.linspace(0, big_pages - 1, c.num_pages).astype(np.int32)[::-1].copy()   # first pages to the top
    table = np.where(c.table >= 0, to[np.maximum(c.table, 0)], -1).astype(np.int32)
    where = torch.from_numpy(to).long().cuda()
    pool = [torch.empty(2, big_pages, HKV, P, D, dtype=ref.TORCH[io], device="cuda") for _ in range(2)]
    assert pool[0].numel() > 2 ** 31
    for x, y in zip(pool, (small.k, small.v)):
        x[:, where] = y
    slots = torch.from_numpy(c.slots).cuda()

    def cache():
        return binding.KvCache(2, big_pages, HKV, P, D, len(c.lens), table.shape[1], io, tensors={
            "k": pool[0], "v": pool[1], "page_table": torch.from_numpy(table).cuda(),
            "n_pages": torch.from_numpy(c.n_pages).cuda(), "length": torch.from_numpy(c.lens).cuda()})

    big = cache()
    c.cache = big
    got, gl = c.call()
    assert binding.kv_read_status(big) == 0 and torch.equal(got, want) and torch.equal(gl, wl)
    # the window's append and the move of an accepted path, in both pools
    plan = binding.RopePlan(D, 64)
    r = np.random.default_rng(16)
    qkv = ref.draw(r, (3, T, HQ + 2 * HKV, D), io).cuda()
    path = torch.tensor([[0, 2, 4, 0, 0], [1, 3, 0, 0, 0], [0, 1, 2, 4, 0]], dtype=torch.int32, device="cuda")
    acc = torch.tensor([3, 2, 4], dtype=torch.int32, device="cuda")
    for cc in (small, big):
        binding.rope_append(plan, cc, 1, slots, qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HKV], qkv[:, :, HQ + HKV:])
        binding.kv_commit(cc, slots, acc, T, path)
        assert binding.kv_read_status(cc) == 0
    for x, y in zip(pool, (small.k, small.v)):
        assert torch.equal(x[:, where], y)
    assert torch.equal(big.length, small.length)
