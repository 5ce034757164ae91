"""Fp4Linear's x far below the largest element of its 128 columns.

Tolerances.  A lone product of an x that f16 holds under its block's power of
two is exact: 0.  Below that the error of x is half a step of f16's
subnormals, 2^-25, against a largest element in [2^14, 2^15): 2^-39 of the
largest element's power of two."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


@pytest.mark.parametrize("top", [2.0 ** 14, 2.0 ** 14 * 1.9921875, 1.0, 2.0 ** 60])
def test_small_elements_beside_a_large_one(m, top):
    """One column's weight is 1, the others' 0: y is x there as f16 held it.  Its bits survive down to 2^-31 of the block's
    largest power of two; below, the error is at most 2^-39 of that."""
    K = 128
    w = torch.zeros(1, K // 2, dtype=torch.uint8)
    w[0, 3] = 0x02                                                # column 6
    op = m.Fp4Linear(K, 1, out_dtype=F32, device=DEV)
    op.transform_weights(w.to(DEV), torch.full((1, K // 32), 127, dtype=torch.uint8, device=DEV))
    unit = 2.0 ** math.floor(math.log2(top))
    for e in range(0, 45):
        for mant in (1.0, 1.9921875, 1.328125):                   # 8 bits each
            v = mant * unit * 2.0 ** -e
            if v > top:
                continue
            x = torch.zeros(1, K, dtype=BF, device=DEV)
            x[0, 100], x[0, 6] = top, v
            assert x[0, 6].item() == v and x[0, 100].item() == top
            err = abs(op.forward(x).item() - v)
            assert err == 0 if e <= 31 else err <= 2.0 ** -39 * unit, (e, mant, err)
