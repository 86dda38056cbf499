"""Forks of a slot whose page table holds an entry that is not a page: the row is refused as a whole,
nothing is shared, copied or handed out for it."""
import pytest

from gated_delta_rule_spec_gb300 import binding
from tests.test_gpu_kv_pages import Both, dev

pytestmark = pytest.mark.gpu


def sources(max_pages, rows, seed=1):
    """A cache with a source of 83 tokens, one of 48 (whole pages), one of 5 and one without any, and
    `rows` empty slots."""
    b = Both(seed, 2, 24, 2, 16, 32, 4 + rows, max_pages, "bf16")
    b.reserve([0, 1, 2], 96, [96, 60, 20])
    for s, n in ((0, 83), (1, 48), (2, 5)):
        b.commit([s], 96, [list(range(n))])
    return b


def spoil(b, slot, col, page):
    """Puts `page` where the slot's table holds another; a function puts that one back."""
    old = int(b.cache.page_table[slot, col])
    b.cache.page_table[slot, col] = page

    def mend():
        b.cache.page_table[slot, col] = old
    return mend


@pytest.mark.parametrize("max_pages,rows", [(6, 5), (20000, 5)])   # tables looked at by one block, and by many
@pytest.mark.parametrize("page", [-1, 24, 2147483647, -2147483648])
@pytest.mark.parametrize("col", [0, 3, 5])                          # 5: the page that is in part filled
def test_fork_of_a_source_with_a_bad_page(max_pages, rows, page, col):
    b = sources(max_pages, rows)
    mend = spoil(b, 0, col, page)
    # to the model the refused row is a padding row: it lacks no page
    done = binding.kv_fork(b.cache, dev([1, 0, 2, 3, 0]), dev([4, 5, 6, 7, 8]))
    want, copies = b.ref.fork([1, -1, 2, 3, -1], [4, 5, 6, 7, 8])
    assert done.tolist() == want == [1, 0, 1, 1, 0]
    assert binding.kv_read_status(b.cache) == binding.ST_PAGE_OOR
    for x in (b.k, b.v):
        for p, q, n in copies:
            x[:, q, :, :n] = x[:, p, :, :n]
    mend()
    b.check()
    b.fork([0], [5])                                                # and once more, now that it is whole
    b.check()
    assert binding.kv_read_status(b.cache) == 0


def test_fork_with_a_bad_page_asks_for_none():
    """One page is left: the spoilt row before it does not use it up; a bad entry behind the committed
    tokens, or beyond the slot's pages, is of no account."""
    b = sources(6, 3)
    b.reserve([4], 96 + 0)                                          # 6 pages more: 6 + 4 + 2 + 6 of 24
    b.reserve([3], 80)                                              # 23 of 24
    mend = spoil(b, 0, 2, 99)
    done = binding.kv_fork(b.cache, dev([0, 2]), dev([5, 6]))
    want, copies = b.ref.fork([-1, 2], [5, 6])
    assert done.tolist() == want == [0, 1] and binding.kv_read_status(b.cache) == binding.ST_PAGE_OOR
    for x in (b.k, b.v):
        for p, q, n in copies:
            x[:, q, :, :n] = x[:, p, :, :n]
    mend()
    b.check()
    b.free([4, 6])
    behind = [spoil(b, 1, 3, 77), spoil(b, 2, 1, -5), spoil(b, 2, 4, 3000)]
    b.fork([1, 2], [4, 6])                                          # 48 tokens in 3 of 4 pages, 5 in 1 of 2
    for mend in behind:
        mend()
    b.check()
    assert binding.kv_read_status(b.cache) == 0


def test_many_forks_some_of_them_bad():
    """More rows than the allocating block has threads."""
    for max_pages, P in ((5, 32), (64, 16)):
        rows = 1100
        b = Both(3, 1, 1400, 1, P, 8, 4 + rows, max_pages, "bf16")
        b.reserve([0, 1, 2, 3], 100)
        for s, n in ((0, 100), (1, 33), (2, 64), (3, 1)):
            b.commit([s], 100, [list(range(n))])
        mend = spoil(b, 1, 1, 1400)
        src = [int(x) for x in b.rng.integers(0, 4, rows)]
        dst = [4 + i for i in range(rows)]
        done = binding.kv_fork(b.cache, dev(src), dev(dst))
        want, copies = b.ref.fork([-1 if s == 1 else s for s in src], dst)
        assert done.tolist() == want == [int(s != 1) for s in src]
        assert binding.kv_read_status(b.cache) == binding.ST_PAGE_OOR
        for x in (b.k, b.v):
            for p, q, n in copies:
                x[:, q, :, :n] = x[:, p, :, :n]
        mend()
        b.check()
