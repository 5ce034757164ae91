"""Scales of the norm's FP8 output are the f32 quotient amax / 448, as the
expert layer's own quantiser has them.  With an f32 stream the normed output
is the very value that is quantised, so scales are compared bit for bit, and
codes are checked against it: q = v / sf rounded to E4M3, where a value that
near a tie may fall on either side (v times the rounded 448 / amax is within
2^-22 of the quotient)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


@pytest.mark.parametrize("T,H", [(300, 128), (300, 512), (64, 1024), (500, 4096), (40, 8320)])
@pytest.mark.parametrize("pad", [0, 1])
def test_scale_is_the_quotient(m, T, H, pad):
    g = torch.Generator().manual_seed(H)
    x = torch.randn(T, H + pad, generator=g)
    x[T // 2:] *= torch.exp(3 * torch.randn(T - T // 2, 1, generator=g))
    x[3] = 0
    x = x.to(DEV)[:, :H]
    w = torch.exp(2 * torch.randn(H, generator=g)).to(DEV)
    w[:128] = 2.0 ** -130 * (1 + torch.arange(128, device=DEV))   # scales among the subnormal floats
    out = m.BlockNorm(H, quant="fp8", dtype=torch.float32, device=DEV).forward(x, w_pre=w)
    v = out.n.cpu().reshape(T, H // 128, 128)
    amax = v.abs().amax(2)
    sf = out.sf.cpu()
    assert torch.equal(sf, amax / torch.tensor(448.0))
    codes = out.codes.cpu().view(torch.float8_e4m3fn).double().reshape(v.shape)
    exact = torch.where(amax[..., None] > 0, v.double() * 448 / amax.double()[..., None], 0.0)
    step = torch.exp2(torch.floor(torch.log2(exact.abs().clamp_min(2.0 ** -6))) - 3)
    assert ((codes - exact).abs() <= step * (0.5 + 2.0 ** -17)).all()


def test_scales_of_extreme_groups(m):
    """A group that overflows has the scale infinity, one of zeros has 0, their neighbours have their own."""
    H = 512
    x = torch.ones(4, H, device=DEV)
    w = torch.ones(H, device=DEV)
    w[5], w[128:256] = torch.inf, 0.0
    w[300] = 3.0e38
    out = m.BlockNorm(H, eps=1e-20, quant="fp8", dtype=torch.float32, device=DEV).forward(x, w_pre=w)
    amax = out.n.cpu().reshape(4, 4, 128).abs().amax(2)
    assert torch.equal(out.sf.cpu(), amax / torch.tensor(448.0))
    assert (out.sf[:, 0] == torch.inf).all() and (out.sf[:, 1] == 0).all() and (out.codes[:, 128:256] == 0).all()
