"""What the packed prompts' calls allocate for themselves on a stream of their own comes from that stream's pool, and a
tensor of another device than the current one is refused; the library, streams and checks are stand-ins."""
import pytest
import torch

from gated_delta_rule_spec_gb300 import binding
from tests.test_binding_streams import FakeStream, Watch


def calls(w, plan):
    norm, starts = binding.HeadNorm(torch.zeros(64)), torch.zeros(3, dtype=torch.int32)
    x, pos = w.q[0], torch.zeros(3, dtype=torch.int32)
    work = torch.zeros(64, dtype=torch.uint8)
    u8, f32, bf16 = torch.uint8, torch.float32, torch.bfloat16
    return [
        (lambda s: binding.norm_rope(plan, norm, pos, x, stream=s), [((3, 4, 64), bf16)]),
        (lambda s: binding.norm_rope_grad(plan, norm, pos, x, x, workspace=work, stream=s), [((3, 4, 64), bf16), ((64,), f32)]),
        (lambda s: binding.norm_rope_grad(plan, norm, pos, x, x, dx=x, dw=norm.weight, stream=s), [((16,), u8)]),
        (lambda s: binding.norm_rope_append(plan, w.cache, 0, w.slots, starts, x, x, x, stream=s), [((3, 4, 64), bf16)]),
        (lambda s: binding.prompt_attn(w.cache, 0, w.slots, starts, x, workspace=work, stream=s), [((3, 4, 64), bf16)]),
        (lambda s: binding.prompt_attn(w.cache, 0, w.slots, starts, x, out=x, stream=s), [((16,), u8)])]


@pytest.mark.parametrize("which", range(6))
def test_results_and_workspaces_are_taken_where_the_call_runs(monkeypatch, which):
    plan = binding.RopePlan(64)                                             # by the library itself
    w, s = Watch(monkeypatch), FakeStream()
    call, made = calls(w, plan)[which]
    call(s)
    assert [(shape, dtype, s) for shape, dtype in made] == w.made
    results = [shape for shape, dtype in made if dtype != torch.uint8]
    assert w.noted == [(shape, "current") for shape in results]            # read there by the caller, perhaps
    w.made.clear(), w.noted.clear()
    call(None)
    assert [(shape, dtype, None) for shape, dtype in made] == w.made and not w.noted


def test_another_device_is_refused(monkeypatch):
    class Elsewhere:
        is_cuda, device = True, "cuda:1"

        def get_device(self):
            return 1

    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    with pytest.raises(binding.GdnSpecError, match="x is on cuda:1"):
        binding._here(x=Elsewhere())


def test_every_tensor_of_a_call_is_looked_at(monkeypatch):
    """Each tensor that a call takes, on another device than the current one in turn."""
    class Somewhere(torch.Tensor):
        is_cuda, at = True, 0

        def get_device(self):
            return self.at

    plan, w = binding.RopePlan(64), Watch(monkeypatch)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    t = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype).as_subclass(Somewhere)  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    norm, k_norm = binding.HeadNorm(t(64, dtype=f32)), binding.HeadNorm(t(64, dtype=f32))
    x, dy, dx, k, v, out = (t(3, 4, 64) for _ in range(6))
    pos, starts, slots = t(3, dtype=i32), t(3, dtype=i32), t(2, dtype=i32)
    dw, lse, work = t(64, dtype=f32), t(3, 4, dtype=f32), t(64, dtype=torch.uint8)
    w.cache.k = t(1)
    for call, tensors in (
            (lambda: binding.norm_rope(plan, norm, pos, x, out=out), (norm._weight, pos, x, out)),
            (lambda: binding.norm_rope_grad(plan, norm, pos, x, dy, dx, dw, work), (norm._weight, pos, x, dy, dx, dw, work)),
            (lambda: binding.norm_rope_append(plan, w.cache, 0, slots, starts, x, k, v, norm, k_norm, pos, out),
             (w.cache.k, slots, starts, x, k, v, norm._weight, k_norm._weight, pos, out)),
            (lambda: binding.prompt_attn(w.cache, 0, slots, starts, x, out=out, lse=lse, workspace=work),
             (w.cache.k, slots, starts, x, out, lse, work))):
        call()
        for one in tensors:
            one.at = 1
            with pytest.raises(binding.GdnSpecError, match="the current device is cuda:0"):
                call()
            one.at = 0


@pytest.mark.parametrize("change", [lambda w: w.to(torch.bfloat16), lambda w: w[:32], lambda w: w.double(), lambda w: w])
def test_a_norms_weights_are_checked_again(change):
    """Converting a model replaces a parameter's memory under the norm that holds it."""
    class Weight(torch.Tensor):
        is_cuda = True

    plan, w = binding.RopePlan(64), torch.zeros(64).as_subclass(Weight)
    norm = binding.HeadNorm(w)
    binding._norm_of(norm, plan, "norm")
    w.data = change(w.data)
    if w.dtype == torch.float32 and w.shape == (64,):
        w.is_cuda = False                                                   # moved to the host
    with pytest.raises(binding.GdnSpecError, match="norm: want contiguous CUDA torch.float32 \\(64,\\)"):
        binding._norm_of(norm, plan, "norm")


def test_a_norms_weights_may_move(monkeypatch):
    """A parameter whose memory is replaced (as by loading or moving a model): the next call reads the new one."""
    plan = binding.RopePlan(64)
    Watch(monkeypatch)
    w = torch.zeros(64)
    norm = binding.HeadNorm(w)
    w.data = torch.ones(64)
    binding._norm_of(norm, plan, "norm")
    assert norm.desc().weight == w.data_ptr()
