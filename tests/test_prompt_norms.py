"""What is given in place of a head norm, without a GPU: the binding looks at it before anything else."""
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding


@pytest.mark.parametrize("bad", [None, torch.ones(64), 1e-6, binding.HeadNormDesc(1 << 20, 1e-6, 0.0)])
def test_no_head_norm(bad):
    plan, pos, x = binding.RopePlan(64), torch.arange(4, dtype=torch.int32), torch.ones(4, 2, 64)
    for call in (lambda: binding.norm_rope(plan, bad, pos, x), lambda: binding.norm_rope_grad(plan, bad, pos, x, x)):
        with pytest.raises(binding.GdnSpecError, match="norm: want a HeadNorm"):
            call()


@pytest.mark.parametrize("side", ["q_norm", "k_norm"])
def test_no_head_norm_of_an_append(side):
    """None is a side without a norm there; anything else that is no HeadNorm is refused by its name."""
    i, x = torch.zeros(2, dtype=torch.int32), torch.ones(4, 2, 64)
    with pytest.raises(binding.GdnSpecError, match=side + ": want a HeadNorm or None"):
        binding.norm_rope_append(binding.RopePlan(64), None, 0, i[:1], i, x, x, x, **{side: torch.ones(64)})
