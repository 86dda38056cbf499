"""A bitmap of free pages that a caller filled, with bits past the last page: such pages are not
handed out, and nothing is written past the pages' counts (here the front of a longer tensor)."""
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [1, 31, 33, 40, 95, 32 * 1024 + 5, 64 * 1024 + 31])
def test_bits_past_the_last_page(pages):
    words = (pages + 31) // 32
    refs = torch.full((words * 32,), 77, dtype=torch.int32, device="cuda")
    refs[:pages] = 0
    cache = binding.KvCache(1, pages, 1, 16, 8, 3, pages + 1, tensors={
        "ref": refs[:pages], "free_bits": torch.full((words,), -1, dtype=torch.int32, device="cuda")})
    slots = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    first = pages // 2
    n = torch.tensor([16 * first, 16 * (pages - first), 16], dtype=torch.int32, device="cuda")
    done = binding.kv_reserve(cache, slots, 16 * pages, n)
    assert done.tolist() == [1, 1, 0] and binding.kv_read_status(cache) == binding.ST_NO_PAGES
    held = torch.cat([cache.page_table[0, :first], cache.page_table[1, :pages - first]])
    assert torch.equal(held, torch.arange(pages, dtype=torch.int32, device="cuda"))
    assert bool((refs[:pages] == 1).all()) and bool((refs[pages:] == 77).all())
    # a fork with a partly filled page finds none either, and one page when one comes back
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    binding.kv_commit(cache, one, torch.tensor([3], dtype=torch.int32, device="cuda"), 3)
    assert binding.kv_fork(cache, one, one + 1).tolist() == [0]
    assert binding.kv_read_status(cache) == binding.ST_NO_PAGES
    if first:
        binding.kv_free(cache, one - 1)
        assert binding.kv_fork(cache, one, one + 1).tolist() == [1]
        assert int(cache.page_table[2, 0]) == 0 and binding.kv_read_status(cache) == 0
    assert bool((refs[pages:] == 77).all())
