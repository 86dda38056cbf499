"""The softmax-attention layers' examples: the C one compiles against the header with
warnings as errors (no link, no GPU), the Python one runs on a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_c_example_compiles(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    inc = os.path.join(ROOT, "include")
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-c", "-I", inc,
                        os.path.join(inc, "gdn_spec_attn_example.c"), "-o", str(tmp_path / "example.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(HQ=6, HKV=3, D=128, P=32, prompts=(1, 130, 64, 65))])
def test_tree_equals_sequential_decoding(kw):
    """Two layers: the tree's outputs on the accepted path are the sequential ones up to bf16 roundings.
    Activations are some 4 at most; each of the two layers rounds its projections, probabilities,
    outputs and residual to bf16 (2^-8 of the value each), which leaves a few times 2^-8 of 4."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import hybrid_tree_step
    finally:
        sys.path.pop(0)
    assert hybrid_tree_step.main(**kw) <= 8 * 4 * 2.0 ** -8
