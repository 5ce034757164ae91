"""An added input that overlaps the output without being it is refused before anything reaches a GPU: tiles are read and stored in no
fixed order.  The output itself, and columns of the same rows beside it, are not (there is only no GPU here, or the call is made)."""
import math

import pytest
import torch

from test_fp8_refusals import BAD, P, backward_input, backward_weight, forward, m  # noqa: F401

ROW = 520 * 2   # bytes of a row of bf16 outputs


@pytest.mark.parametrize("T,add,y,ld_add,ld_y", [
    (4, P + ROW, P, 520, 520), (4, P, P + ROW, 520, 520), (4, P + 3 * ROW, P, 520, 520), (4, P, P + 3 * ROW, 520, 520),   # rows before or after
    (4, P + 512, P, 520, 520), (4, P, P + 512, 520, 520), (4, P + 1024, P, 1024, 1024 - 8),                             # columns that meet
    (2, P + 512, P, 1024, 1024), (4, P + 1536, P, 1024, 1024), (4, P, P + 1536, 1024, 1024),
    (1, P + 16, P, 512, 512), (1, P, P + 1008, 4096, 520),                                                               # one row
    (4, P + 2 * 520, P, 1040, 520), (4, P, P + 2 * 1040, 520, 1040), (4, P + 16, P, 528, 520)])                         # other pitches
def test_refused(m, T, add, y, ld_add, ld_y):  # noqa: F811
    c = m.Fp8LinearConfig(256, 512, 0, 0, 0, math.inf)
    assert forward(m, c, T=T, add=add, ld_add=ld_add, y=y, ld_y=ld_y) == BAD
    i = m.Fp8LinearConfig(512, 256, 0, 0, 0, math.inf)
    assert backward_input(m, i, T=T, ld_dy=256, add=add, ld_add=ld_add, dx=y, ld_dx=ld_y) == BAD
    w = m.Fp8LinearConfig(256, 16 * T, 0, 0, 0, math.inf)   # f32: a row of 256 is as long
    assert backward_weight(m, w, T=4, ld_dy=16 * T, add=P + 256 * 4, ld_add=256, dw=P, ld_dw=256) == BAD
    assert backward_weight(m, w, T=0, ld_dy=16 * T, add=P + 256 * 4, ld_add=256, dw=P, ld_dw=256) == BAD


@pytest.mark.parametrize("T,add,y,ld_add,ld_y", [
    (4, P, P, 520, 520), (1, P, P, 520, 528),                                            # the output
    (4, P + 3 * ROW + 1024, P, 520, 520), (4, P, P + 4 * ROW, 520, 520),                 # behind it
    (4, P + 1024, P, 1024, 1024), (4, P, P + 1024, 1024, 1024), (4, P + 1040, P, 1040, 1040),   # columns beside it
    (4, P + 1040, P, 1040, 1040), (4, P + 3 * ROW + 1024, P, 4096, 520),
    (1, P + 1024, P, 512, 512)])
def test_not_refused(m, T, add, y, ld_add, ld_y):  # noqa: F811
    """Calls that the checks let pass reach the device, of which there must be none: they are made on the CPU alone."""
    if torch.cuda.is_available():
        pytest.skip("pointers of this test are no memory")
    c = m.Fp8LinearConfig(256, 512, 0, 0, 0, math.inf)
    assert forward(m, c, T=T, add=add, ld_add=ld_add, y=y, ld_y=ld_y) == -3
    i = m.Fp8LinearConfig(512, 256, 0, 0, 0, math.inf)
    assert backward_input(m, i, T=T, ld_dy=256, add=add, ld_add=ld_add, dx=y, ld_dx=ld_y) == -3
