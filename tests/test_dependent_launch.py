"""Reading the kernels' source: what a kernel that is launched dependently owes the one before it
and the one behind it, on every way out.

Such a kernel may start while the one before it still runs, and a block that has ended counts as
one that has let the next launch go, so a block that left without waiting could let the next kernel
run beside the one before.  And the kernel that joins split rows reads a note from every chunk."""
import glob
import os
import re

import pytest

from gated_delta_rule_spec_gb300 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu")))


def plain(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def body(text, at):
    """The braces' contents from the first one behind `at`."""
    i = text.index("{", at)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError("unbalanced braces")


def kernels():
    """(file, name, body) of every kernel that some launch_dependent names."""
    text = {p: plain(open(p).read()) for p in SOURCES}
    launched = {m for t in text.values() for m in re.findall(r"launch_dependent\(\s*(\w+)", t)} - {"kern"}
    for p, t in text.items():
        for m in re.finditer(r"__global__", t):
            name = re.search(r"(\w*_kernel)\s*\(", t[m.end():]).group(1)
            if name in launched:
                yield os.path.basename(p), name, body(t, m.end() + t[m.end():].index(name + "("))


FOUND = list(kernels())


def test_the_kernels_are_found():
    assert {"kv_alloc_kernel", "rope_kernel", "tree_attn_kernel", "tree_attn_tc_kernel", "attn_join_kernel"} <= {
        n for _, n, _ in FOUND}


@pytest.mark.parametrize("file,name,code", FOUND, ids=[n for _, n, _ in FOUND])
def test_every_way_out_is_behind_the_wait(file, name, code):
    wait = code.index("grid_dep_wait()")
    for way in (r"\breturn\b", r"grid_dep_launch\(\)", r"atomic\w+\("):
        at = re.search(way, code)
        assert at is None or at.start() > wait, (file, name, way)


def test_a_block_that_gives_up_early_leaves_the_join_a_note():
    code = next(c for _, n, c in FOUND if n == "tree_attn_tc_kernel")
    way_out = code[:code.index("return")]
    assert re.search(r"attn_note\(A, group, false,", way_out)
    common = plain(open(os.path.join(build.CSRC, "attn_common.cuh")).read())
    assert re.search(r"AttnCut\{-1,", body(common, common.index("void attn_note")))
    join = next(c for _, n, c in FOUND if n == "attn_join_kernel")
    assert join.index("cut.b < 0") < join.index("/ cut.chunk")      # an empty chunk is left before its size is used
