"""The cache's pages at the sizes of a whole model's cache: moves of more columns than one block a
row takes, copies of long parts of pages, grids smaller than their work.  The model and the
comparison, bit for bit after every call, are those of test_gpu_kv_pages.py."""
import pytest

from gated_delta_rule_spec_gb300 import binding
from tests.test_gpu_kv_pages import Both

pytestmark = pytest.mark.gpu


def paths(r, n, T):
    return [sorted(int(x) for x in r.permutation(T)[:int(r.integers(1, T + 1))]) for _ in range(n)]


def lives(b, T, rounds):
    """Prompts of odd lengths, forks, and steps of reserve, commit with a path and free."""
    r, slots = b.rng, len(b.ref.pages)
    first = list(range(slots // 2))
    counts = [int(x) for x in r.integers(1, T + 1, len(first))]
    b.reserve(first, T, counts)
    b.check()
    b.commit(first, T, [list(range(n)) for n in counts])
    b.check()
    for _ in range(rounds):
        dst = [s for s in range(slots) if not b.ref.pages[s]][:len(first)]
        b.fork([int(r.choice(first)) for _ in dst], dst)
        b.check()
        rows = [int(s) for s in r.permutation(first + dst)]
        rows = [s for s in rows if -(-(b.ref.length[s] + T) // b.ref.P) <= b.ref.max_pages]
        b.reserve(rows, T)
        b.check()
        b.commit(rows, T, paths(r, len(rows), T))
        b.check()
        b.free(dst)
        b.check()
    assert binding.kv_read_status(b.cache) == 0


@pytest.mark.parametrize("io,layers,HKV,P,D", [("bf16", 12, 2, 64, 256), ("fp32", 9, 3, 128, 96)])
def test_a_models_cache(io, layers, HKV, P, D):
    """1536 and 1296 columns of 16 bytes a token: the move has six blocks a row and the advance a launch
    of its own; parts of pages of up to 2016 and 3048 pieces a head."""
    assert layers * HKV * 2 * (D * (2 if io == "bf16" else 4) // 16) > 4 * 256
    lives(Both(21, layers, 40, HKV, P, D, 8, 5, io), T=P - 1, rounds=3)


def test_more_rows_than_the_grids_have_blocks():
    """Forks of 60 rows with 192 runs each on 137 blocks a row; moves of 120 rows with 3072 columns each on
    11 blocks of 256."""
    b = Both(22, 12, 520, 8, 16, 128, 120, 8, "bf16")
    assert -(-8192 // 60) < 12 * 8 * 2 and -(-1280 // 120) * 256 < 12 * 8 * 2 * 16
    lives(b, T=16, rounds=2)
