"""An added input that starts where the output does is the output: rows of another pitch are refused before anything reaches a GPU.  And the
sources' shared parts, whose kernels start early too, have no non-coherent loads."""
import glob
import math
import os
import re

import pytest

from test_early_start_loads import CSRC, NON_COHERENT
from test_fp8_refusals import BAD, P, backward_input, backward_weight, forward, m  # noqa: F401


def test_the_output_with_another_pitch(m):  # noqa: F811
    c = m.Fp8LinearConfig(256, 512, 0, 0, 0, math.inf)
    assert forward(m, c, add=P, ld_add=520, ld_y=512) == BAD
    assert backward_input(m, c, add=P, ld_add=264, ld_dx=256) == BAD
    assert backward_weight(m, c, add=P, ld_add=260, ld_dw=256) == BAD
    assert backward_weight(m, c, T=0, add=P, ld_add=260, ld_dw=256) == BAD


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cuh"))), ids=os.path.basename)
def test_no_non_coherent_loads_in_shared_parts(path):
    code = re.sub(r"//[^\n]*", "", open(path).read())
    if "wait_for_previous()" in code:
        assert not NON_COHERENT.search(code)
