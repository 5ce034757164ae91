"""Products that are no numbers, or infinite, through SwiGLU and its clamp."""
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


@pytest.mark.parametrize("clamp", [4.0, math.inf])
@pytest.mark.parametrize("M", [1, 3, 9])
def test_nan_goes_through_swiglu(m, M, clamp):
    """A NaN in x makes its token's outputs NaN, clamped or not, and no other token's."""
    N, K = 48, 256
    g = torch.Generator().manual_seed(M)
    w = (torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8) | 0x11).to(DEV)
    sf = torch.full((N, K // 32), 125, dtype=torch.uint8, device=DEV)
    op = m.Fp4Linear(K, N, act="swiglu", act_clamp=clamp, out_dtype=F32, device=DEV)
    op.transform_weights(w, sf)
    x = torch.randn(M, K, generator=g).to(BF).to(DEV)
    clean = op.forward(x)
    x[M // 2, 77] = math.nan
    out = op.forward(x)
    assert torch.isnan(out[M // 2]).all()
    keep = [i for i in range(M) if i != M // 2]
    assert torch.equal(out[keep], clean[keep]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("half", ["gate", "up"])
def test_nan_in_one_half(m, half):
    """A NaN that only the gate's or only the up half's weights see: infinity times a zero code."""
    N, K = 32, 128
    w = torch.full((N, K // 2), 0x22, dtype=torch.uint8)          # all 1.0
    rows = slice(0, 16) if half == "gate" else slice(16, 32)
    w[rows, 5] = 0x20                                             # column 10: code 0, so that inf * 0 is NaN there
    sf = torch.full((N, K // 32), 127, dtype=torch.uint8)
    op = m.Fp4Linear(K, N, act="swiglu", act_clamp=7.0, out_dtype=F32, device=DEV)
    op.transform_weights(w.to(DEV), sf.to(DEV))
    x = torch.ones(1, K, dtype=BF, device=DEV)
    x[0, 10] = math.inf
    assert torch.isnan(op.forward(x)).all()


def test_infinities_clamp(m):
    """An infinite product is a number once clamped: silu(c) c, and a gate of -c."""
    N, K, c = 32, 128, 7.0
    w = torch.full((N, K // 2), 0x22, dtype=torch.uint8)
    op = m.Fp4Linear(K, N, act="swiglu", act_clamp=c, out_dtype=F32, device=DEV)
    op.transform_weights(w.to(DEV), torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV))
    x = torch.ones(2, K, dtype=BF, device=DEV)
    x[0, 10], x[1, 10] = math.inf, -math.inf
    out = op.forward(x).double().cpu()
    for row, v in ((0, c), (1, -c)):
        want = v / (1 + math.exp(-v)) * v
        assert ((out[row] - want).abs() <= 2.0 ** -20 * abs(want)).all()
