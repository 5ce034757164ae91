"""Kernels that may be set up while the one before them runs
(wait_for_previous) share the GPU with the writer of what they will read.  The
non-coherent load is for memory that nobody writes while a kernel is resident:
their sources have none, in any of its spellings."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_ffn_gb300", "csrc")
NON_COHERENT = re.compile(r"__ldg\b|\.global(\.[\w:]+)*\.nc\b|\b__restrict(__)?\b|\btex1Dfetch\b")


def early():
    return [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "wait_for_previous()" in open(f).read()]


def test_there_are_some():
    assert {os.path.basename(f) for f in early()} >= {"moe_norm.cu", "moe_router.cu", "moe_linear.cu"}


@pytest.mark.parametrize("path", early() + [os.path.join(CSRC, "moe_ops.cuh")], ids=os.path.basename)
def test_no_non_coherent_loads(path):
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert not NON_COHERENT.search(code), NON_COHERENT.search(code)
