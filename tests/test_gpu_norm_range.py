"""BlockNorm.backward where the cube of the reciprocal root leaves the f32
range: rows of very large or very small magnitude, rows of zeros under a tiny
eps.

Tolerance.  Every factor of a gradient is in range (checked on the 64-bit
reference: no term above 2^126), so its error is that of its roundings: 2^-20
of the sum of its terms' magnitudes, one rounding of the output (2^-23 f32,
2^-8 bf16), and 2^-126 for values that are subnormal."""
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


def reference(h, dn, w, eps):
    """D of the pre norm alone, and the magnitude of its terms."""
    h, dn, w = h.double().cpu(), dn.double().cpu(), w.double().cpu()
    r = (h.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    a, hat = dn * w, h * r
    back = hat * (a * hat).mean(1, keepdim=True)
    return r, r * (a - back), r * (a.abs() + hat.abs() * (a * hat).abs().mean(1, keepdim=True))


def check(m, h, dn, w, eps, dtype):
    r, ref, mag = reference(h, dn, w, eps)
    assert max(r.max(), mag.max()) < 2.0 ** 126
    op = m.BlockNorm(h.shape[1], float(eps), dtype=dtype, device=DEV)
    fwd = op.forward(h, w_pre=w)
    got = op.backward(h, dn=dn, w_pre=w, rstd_pre=fwd.rstd_pre).dresidual.double().cpu()
    u = 2.0 ** -8 if dtype == BF else 2.0 ** -23
    err = (got - ref).abs()
    tol = u * ref.abs() + 2.0 ** -20 * mag + 2.0 ** -126
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.3g} x tolerance"


# the variants: a warp's and CTAs' rows, chunks a thread, by element, over 8192 columns; many rows: two a pass
SHAPES = [(5, 64), (7, 1000), (7, 1001), (400, 4096), (3, 5001), (2, 8320), (2, 16384), (700, 2048)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("power", [-55, -40, 37, 42, 46, 50])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_rows_of_any_magnitude(m, T, H, power, dtype):
    """dn along h, where the two terms of the gradient cancel, and dn at random; the mean of squares stays within f32."""
    g = torch.Generator().manual_seed(H + power)
    x = torch.randn(T, H, generator=g)
    h = torch.ldexp(x, torch.tensor(power)).to(dtype).to(DEV)
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(DEV)
    eps = 2.0 ** -120
    for dn in (torch.randn(T, H, generator=g).to(dtype).to(DEV), x.to(dtype).to(DEV)):
        check(m, h, dn, w, eps, dtype)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("eps", [1e-6, 1e-27, 1e-30, 1e-37])
def test_rows_of_zeros(m, T, H, eps):
    """A padding row's gradient is r dn w: large, but a number."""
    g = torch.Generator().manual_seed(T)
    h = torch.zeros(T, H, device=DEV)
    h[1::2] = torch.randn(h[1::2].shape, generator=g).to(DEV)
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(DEV)
    check(m, h, torch.randn(T, H, generator=g).to(DEV), w, torch.tensor(eps).item(), F32)
