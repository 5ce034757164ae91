"""Size of the FP4 linear's weight store: a block of 128 columns of 32 rows is
2048 bytes of codes and 128 of scales, and every row has an exponent."""
import math

import pytest


@pytest.fixture(scope="module")
def m():
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 28672, 2 ** 31 - 34, 2 ** 31 - 33, 2 ** 31 - 32, 2 ** 31 - 31, 2 ** 31 - 2, 2 ** 31 - 1])
@pytest.mark.parametrize("k", [32, 128, 160, 24576])
def test_bytes(m, n, k, act):
    if act and n % 2:
        return
    tiles, blocks = -(-n // 32), -(-k // 128)
    up = lambda b: -(-b // 256) * 256  # noqa: E731
    want = up(tiles * blocks * 2176) + up(tiles * 32 * 4)
    assert m.lib().moe_fp4_linear_weight_bytes(m.Fp4LinearConfig(k, n, act, 0, math.inf)) == want
