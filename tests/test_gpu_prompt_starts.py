"""Entries of `starts` that do not ascend inside [0, N], anywhere in the list: which rows own their tokens is the same to
the append and to the attention, and the rows that do are as ever (bounds: prompt_case.py, test_gpu_norm_rope.py)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests import attn_ref as ref
from tests import norm_ref
from tests.prompt_case import HALF_ULP, Prompts, attention

pytestmark = pytest.mark.gpu

FEW = [20, 30, 40, 25]


def many(n):
    return [(i * 7) % 13 for i in range(n)]


def owners(starts, N):
    """Whether each row owns its tokens: it is a range, and none before it that is one reaches past its first token."""
    own, reach = [], 0
    for a, e in zip(starts[:-1], starts[1:]):
        proper = 0 <= a <= e <= N
        own.append(proper and a >= reach)
        if proper:
            reach = max(reach, e)
    return own


# the entries that are replaced, and by what: below all, past the tensors, back among earlier rows, far ahead
LISTS = [(FEW, {2: -3}), (FEW, {1: -1}), (FEW, {2: 10 ** 6}), (FEW, {2: 10}), (FEW, {1: 70}), (FEW, {2: -2 ** 31, 3: 2 ** 31 - 1}),
         (FEW, {3: 20}), (FEW, {0: 20, 1: 0}),
         (many(70), {33: -5}), (many(70), {32: 10 ** 6}), (many(70), {40: 3}), (many(70), {10: 300, 60: 7}),
         (many(70), {31: -1, 32: -1, 33: -1, 64: -1}), (many(700), {31: -7, 400: 2 ** 30}), (many(700), {350: 4000}),
         (many(700), {n: -1 for n in range(0, 701, 22)})]


def case(counts, change, io, D, layers=1, layer=0):
    """A padding row in it, tokens of no row at both ends."""
    B = len(counts)
    slots = [-1 if b % 9 == 3 else b for b in range(B)]
    c = Prompts(41, io, 4, 2, D, 32, counts, [(b * 11) % 71 for b in range(B)], slots=slots, layers=layers, layer=layer,
                poison=False, lead=2, tail=5)
    good = c.starts.copy()
    for at, value in change.items():
        c.starts[at] = value
    own = owners([int(x) for x in c.starts], c.N)
    assert not all(own) and not np.array_equal(good, c.starts)
    return c, own


def rows_of(c, own):
    """(row, first, end, slot, fits) of the rows that own tokens."""
    for b, (a, e) in enumerate(zip(c.starts[:-1].tolist(), c.starts[1:].tolist())):
        if own[b] and a < e:
            s = int(c.slots[b])
            yield b, a, e, s, s >= 0 and int(c.lens[s]) + e - a <= int(c.n_pages[s]) * c.P


def status_of(c, own):
    short = any(s >= 0 and not fits for _, _, _, s, fits in rows_of(c, own))
    return binding.ST_ACCEPT_RANGE | (binding.ST_NO_PAGES if short else 0)


@pytest.mark.parametrize("io,D", [("bf16", 128), ("bf16", 256), ("fp32", 64)])
@pytest.mark.parametrize("n", range(len(LISTS)))
def test_attention(io, D, n):
    c, own = case(*LISTS[n], io, D)
    out, lse = c.call()
    assert binding.kv_read_status(c.cache) == status_of(c, own)
    got, gl, nobodys = out.double().cpu().numpy(), lse.double().cpu().numpy(), np.ones(c.N, bool)
    q, k, v = (x.double().numpy() for x in (c.q, c.k[0], c.v[0]))
    for b, a, e, s, fits in rows_of(c, own):
        nobodys[a:e] = False
        if not fits:   # a padding row, or one whose tokens have no pages
            assert (got[a:e] == 0).all() and np.isneginf(gl[a:e]).all(), b
            continue
        want, wl, spread = attention(q[a:e], k, v, c.table, [s], c.lens, [0, e - a], c.scale)
        assert (np.abs(got[a:e] - want) <= c.bound(want, spread)).all(), b
        assert (np.abs(gl[a:e] - wl) <= 2e-5).all(), b
    assert (got[nobodys] == 7).all() and (gl[nobodys] == 7).all()


@pytest.mark.parametrize("io,D", [("bf16", 128), ("bf16", 40), ("fp32", 64)])
@pytest.mark.parametrize("n", range(len(LISTS)))
def test_append(io, D, n):
    c, own = case(*LISTS[n], io, D, layers=2, layer=1)
    cache = c.upload()
    qkv = ref.draw(c.rng, (c.N, 8, D), io)
    dev, out = qkv.cuda(), torch.full((c.N, 4, D), 7.0, dtype=ref.TORCH[io], device="cuda")
    w = torch.from_numpy((1 + 0.3 * c.rng.standard_normal(D)).astype(np.float32))
    norm = binding.HeadNorm(w.cuda())
    binding.norm_rope_append(binding.RopePlan(D), cache, 1, torch.from_numpy(c.slots).cuda(), torch.from_numpy(c.starts).cuda(),
                             dev[:, :4], dev[:, 4:6], dev[:, 6:], norm, norm, q_out=out)
    assert binding.kv_read_status(cache) == status_of(c, own)
    f, m = ref.frequencies(D)
    x = qkv.double().numpy()
    y = x[:, :6] * norm_ref.root(x[:, :6], np.float64(np.float32(1e-6))) * w.double().numpy()
    got, kg, vg, k1, v1 = out.double().cpu().numpy(), cache.k.cpu(), cache.v.cpu(), c.k.clone(), c.v.clone()
    nobodys = np.ones(c.N, bool)
    for b, a, e, s, fits in rows_of(c, own):
        nobodys[a:e] = False
        if not fits:
            assert (got[a:e] == 0).all(), b
            continue
        i = int(c.lens[s]) + np.arange(e - a)
        want = ref.rotate(y[a:e], i.astype(np.int32), f, m, D, "half")
        bound = 2.0 ** -18 * norm_ref.size(y[a:e], D, "half", m) + HALF_ULP[io] * np.abs(want)
        page, off = torch.from_numpy(c.table[s, i // c.P]).long(), torch.from_numpy(i % c.P)
        key = kg[1, page, :, off]
        assert (np.abs(got[a:e] - want[:, :4]) <= bound[:, :4]).all(), b
        assert (np.abs(key.double().numpy() - want[:, 4:]) <= bound[:, 4:]).all(), b
        k1[1, page, :, off] = key
        v1[1, page, :, off] = qkv[a:e, 6:]
    assert (got[nobodys] == 7).all()
    assert torch.equal(kg, k1) and torch.equal(vg, v1)            # nothing else was written


def test_a_list_that_is_mended_between_replays():
    """The list is read at each replay of a captured step: a bad one spoils nothing for the next."""
    c = Prompts(42, "bf16", 4, 2, 128, 32, FEW, [10, 0, 70, 33], poison=False)
    want, wl = c.check()
    starts, good = torch.from_numpy(c.starts).cuda(), torch.from_numpy(c.starts).cuda()
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    slots, q = torch.from_numpy(c.slots).cuda(), c.q.cuda()
    work = torch.empty(binding.prompt_attn_workspace(c.cache, 4, c.N, 4), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.prompt_attn(c.cache, 0, slots, starts, q, scale=c.scale, out=out, lse=lse, workspace=work)
    for at, value in ((2, -3), (1, 10 ** 6), (3, 5)):
        starts[at] = value
        out.fill_(7.0)
        g.replay()
        assert binding.kv_read_status(c.cache) == binding.ST_ACCEPT_RANGE
        assert (out == 7).any()
        starts.copy_(good)
        g.replay()
        torch.cuda.synchronize()
        assert binding.kv_read_status(c.cache) == 0 and torch.equal(out, want) and torch.equal(lse, wl)
