"""Kernels that start before their predecessor ends (no GPU): what the predecessor writes is changing
while they are resident, so it must not be read as read-only data, by a non-coherent load or
through a pointer that the compiler may take for unaliased."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_varlen_rope_gb300", "csrc")


def early_kernels(name):
    """(kernel, its parameters, its body) of those that wait for their predecessor."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for at in re.finditer(r"__global__ void[^{;]*?\b(\w+_kernel)\(([^{]*)\)\s*\{", text):
        body = text[at.end():]
        body = body[:body.index("\n}")]
        if "griddepcontrol.wait" in body:
            yield at.group(1), at.group(2), body


@pytest.mark.parametrize("name,count", [("attn_fwd.cu", 2), ("attn_bwd.cu", 2), ("attn_decode.cu", 1)])
def test_no_parameter_is_taken_for_unaliased(name, count):
    kernels = list(early_kernels(name))
    assert len(kernels) == count
    for kernel, parameters, _ in kernels:
        assert "__restrict__" not in parameters, kernel


def test_statistics_and_outputs_are_read_coherently():
    """The backward's kernels read what the forward and each other write; offsets and lengths go
    through find_slot."""
    for kernel, _, body in early_kernels("attn_bwd.cu"):
        assert "__ldg" not in body, kernel
    for kernel, _, body in early_kernels("attn_fwd.cu"):
        assert all("a.table" in line for line in body.splitlines() if "__ldg" in line), kernel
