"""Kernels launched as programmatic dependents of a kernel that lets them start early have to wait for it in
every CTA: otherwise their grid can be over while the kernel before still writes, and what follows in the
stream or in a captured graph is ordered behind the dependent grid only.  Read from the sources: no way out of
such a kernel lies before its wait."""

import os
import re

import pytest

from speculative_decoding_verify_attn_gb300.build import CSRC

FILES = ["paged_mma.cu", "chunk_plan.cu", "chunk_tc.cu", "chunk_f32.cu", "logprobs.cu"]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(text):
    """Name -> body of every kernel (up to the next closing brace in the first column)."""
    found = {}
    for m in re.finditer(r"__global__[^;{]*?\b(\w+)\(const __grid_constant__[^{;]*\{", text):
        found[m.group(1)] = text[m.end():text.index("\n}", m.end())]
    return found


def dependents(text):
    names = set(re.findall(r"launch_dependent\((\w+)", text))
    if "kern" in names:  # a variable: what it is set to
        names = (names - {"kern"}) | set(re.findall(r"auto kern = (\w+)", text))
    return names


@pytest.mark.parametrize("name", FILES)
def test_dependent_grids_wait_before_they_leave(name):
    text = source(name)
    bodies, names = kernels(text), dependents(text)
    assert names and names <= set(bodies)
    for k in names:
        before, wait, _ = bodies[k].partition("pdl_wait();")
        assert wait, f"{k} never waits"
        assert "return" not in before, f"{k} can return before its wait"
