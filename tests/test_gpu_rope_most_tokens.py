"""Rotary positions of as many tokens as the call takes: 2^31 - 1 (43 GB, in place)."""
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding

pytestmark = pytest.mark.gpu


def test_the_largest_number_of_tokens():
    n = 2 ** 31 - 1
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("not enough free memory for 2^31 tokens")
    plan = binding.RopePlan(8, 2)
    x = torch.ones(n, 1, 8, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    binding.rope(plan, pos, x, out=x)
    for a in (0, 12345, 2 ** 30 - 500, n - 1000):
        part = slice(a, a + 1000)
        want = binding.rope(plan, pos[part].clone(), torch.ones(1000, 1, 8, dtype=torch.bfloat16, device="cuda"))
        assert torch.equal(x[part], want)
    # no token was left out: pair 0 turns by one radian a token, so both of its values are one for position 0 alone
    step = 1 << 27
    still = sum(int(((x[a:a + step, 0, 0] == 1) & (x[a:a + step, 0, 1] == 1)).sum()) for a in range(0, n, step))
    near = sum(int((torch.remainder(pos[a:a + step].double(), 2 * torch.pi).sub_(torch.pi).abs_() > torch.pi - 0.004).sum())
               for a in range(0, n, step))
    assert still <= near
    del x, pos
    torch.cuda.empty_cache()
