"""The binding's cache object: its calls use the tensors that it holds, also after one was replaced."""
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding

TENSORS = ("k", "v", "page_table", "n_pages", "length", "ref", "free_bits", "status")


def pointers(cache):
    return {n: getattr(cache.desc(), n) for n in TENSORS}


def test_a_replaced_tensor_is_the_one_that_calls_get(monkeypatch):
    cache = binding.KvCache(2, 40, 2, 16, 64, 3, 5, device="cpu")
    assert pointers(cache) == {n: getattr(cache, n).data_ptr() for n in TENSORS}
    kept = cache._ref._obj
    monkeypatch.setattr(binding, "_need", lambda *a: None)        # which asks for CUDA tensors
    for n in TENSORS:
        x = torch.clone(getattr(cache, n))
        setattr(cache, n, x)
        assert getattr(cache, n) is x
        assert pointers(cache) == {m: getattr(cache, m).data_ptr() for m in TENSORS}
    assert cache._ref._obj is kept is cache.desc()


def test_what_does_not_fit_is_refused():
    cache = binding.KvCache(2, 40, 2, 16, 64, 3, 5, device="cpu")
    before, held = pointers(cache), {n: getattr(cache, n) for n in TENSORS}
    for n in TENSORS:
        with pytest.raises(binding.GdnSpecError):
            setattr(cache, n, held[n].clone())                    # not on the GPU
    for n in ("n_layers", "num_pages", "HKV", "P", "D", "num_slots", "max_pages", "io_code", "io_torch"):
        value = getattr(cache, n)
        with pytest.raises(binding.GdnSpecError):
            setattr(cache, n, value)
        assert getattr(cache, n) == value
    assert pointers(cache) == before and all(getattr(cache, n) is held[n] for n in TENSORS)


@pytest.mark.gpu
def test_calls_follow_a_replaced_tensor():
    cache = binding.KvCache(1, 12, 2, 16, 64, 3, 4)
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    old = {n: getattr(cache, n) for n in TENSORS}
    for n in TENSORS:
        setattr(cache, n, old[n].clone())
    assert bool(binding.kv_reserve(cache, slots, 20).all())
    qkv = torch.ones(3, 4, 8, 64, dtype=torch.bfloat16, device="cuda")
    binding.rope_append(binding.RopePlan(64), cache, 0, slots, qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:])
    binding.kv_commit(cache, slots, torch.full((3,), 3, dtype=torch.int32, device="cuda"), 4)
    binding.kv_reserve(cache, slots, 100)                         # more columns than there are
    assert binding.kv_read_status(cache) == binding.ST_NO_PAGES
    assert cache.length.tolist() == [3] * 3 and cache.n_pages.tolist() == [2] * 3
    assert cache.page_table[:, :2].tolist() == [[0, 1], [2, 3], [4, 5]] and cache.ref.tolist() == [1] * 6 + [0] * 6
    assert bool((cache.v[0, [0, 2, 4], :, :4] == 1).all()) and bool((cache.k[0, [0, 2, 4], :, :4] != 0).any())
    assert old["length"].tolist() == [0] * 3 and old["ref"].tolist() == [0] * 12 and bool((old["page_table"] == -1).all())
    for bad in (cache.k.float(), cache.k[:, :6], cache.k.transpose(3, 4), cache.k.cpu()):
        with pytest.raises(binding.GdnSpecError):
            cache.k = bad
    with pytest.raises(binding.GdnSpecError):
        cache.status = cache.status[:0]
