"""Groups whose largest magnitude is so small that amax / 448 rounds to no f32 but zero (below 2^-141): their codes are zeros, their
scale is zero, and no finite input becomes a NaN.  Next to them groups whose scale is the smallest number.

Tolerances: fp8_ref.close_codes, whose 448 * 2^-149 is what a scale below the normal numbers leaves of a value."""
import pytest
import torch

from fp8_ref import BF, DEV, F32, close_codes, up

pytestmark = pytest.mark.gpu
TINY = [-149, -147, -145, -143, -142, -141, -140, -135]


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    yield mod
    assert mod.lib().moe_fp8_linear_status() == mod.MOE_OK


def nans(codes):
    return int(((codes & 127) == 127).sum())


def check(codes, sf, v, br, bc):
    assert nans(codes) == 0
    assert ((codes & 127) == 0)[v == 0].all()
    close_codes(codes, sf, v, torch.zeros_like(v), br, bc)
    amax = torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % bc, 0, -v.shape[0] % br))
    amax = amax.reshape(-(-v.shape[0] // br), br, -(-v.shape[1] // bc), bc).amax((1, 3))
    assert torch.equal(sf, (amax / 448).float())


@pytest.mark.parametrize("T,H", [(8, 144), (130, 144), (1100, 272)])
def test_one_tiny_value_among_zeros(m, T, H):
    """(1100 rows: the form of many rows.)"""
    for e in TINY:
        v = torch.zeros(T, H, device=DEV)
        v[T // 2, H // 2] = 2.0 ** e if T % 4 else -(2.0 ** e)
        v[0, 0] = 3.0 * 2.0 ** -149
        op = m.Fp8Quant(H, dtype=F32, device=DEV)
        o = op.forward(v, cols=True)
        check(o.codes, o.sf, v.double(), 1, 128)
        check(o.col_codes, o.col_sf, v.double(), 128, 1)
        o = op.forward(v)
        check(o.codes, o.sf, v.double(), 1, 128)
        o = op.weights(v)
        check(o.codes, o.sf, v.double(), 128, 128)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 200])
def test_a_saturated_gate_among_zeros(m, T, dt):
    """Gate -95 (a sigmoid of 5.5e-42) in one token among padding: SwiGLU's output and gradient have no NaN, and the weight's
    gradient of such columns is finite."""
    H = 128
    for d0 in (2.0 ** -8, 2.0 ** -10, 2.0 ** -12, 2.0 ** -14):
        v, d = torch.zeros(T, 2 * H, dtype=dt, device=DEV), torch.zeros(T, H, dtype=dt, device=DEV)
        v[3, 7], v[3, H + 7], d[3, 7] = -95.0, d0, d0
        op = m.Fp8Quant(H, act="swiglu", dtype=dt, device=DEV)
        for o in (op.forward(v, cols=True), op.backward(d, v)):
            assert nans(o.codes) == 0 and nans(o.col_codes) == 0
            assert torch.isfinite(o.sf).all() and torch.isfinite(o.col_sf).all()
        o = op.backward(d, v)
        x, x_sf = torch.full((T, 16), 0x38, dtype=torch.uint8, device=DEV), torch.ones(up(T), 16, device=DEV)   # ones
        dw = m.Fp8Linear(16, 2 * H, device=DEV).backward_weight(o.col_codes, o.col_sf, x, x_sf)
        assert torch.isfinite(dw).all()


@pytest.mark.parametrize("T", [3, 40, 700, 30000])
def test_the_linears_codes(m, T):
    """One output column of silu(-95) * 2^-n, the others of the group zero."""
    K, N = 16, 512
    one, minus = 0x38, 0xB8
    x, x_sf = torch.zeros(T, K, dtype=torch.uint8, device=DEV), torch.ones(T, 1, device=DEV)
    x[:, 0] = one
    w = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    w[5, 0], w[N // 2 + 5, 0] = minus, one
    op = m.Fp8Linear(K, N, act="swiglu", quant="fp8", device=DEV)
    for n in (4, 9, 11, 13, 15):
        w_sf = torch.tensor([95.0, 1.0, 2.0 ** -n, 1.0], device=DEV).reshape(4, 1)
        o = op.forward(x, x_sf, w, w_sf)
        y = -95.0 * torch.sigmoid(torch.tensor(-95.0, dtype=torch.float64)) * 2.0 ** -n
        assert nans(o.codes) == 0
        rest = o.codes.clone()
        rest[:, 5] = 0
        assert ((rest & 127) == 0).all() and (o.sf[:, 1] == 0).all()
        # the sigmoid and two products below the normal numbers: 2^-149 each, 95 times the first
        err = 2.0 ** -149 * (95 * 2.0 ** -n + 2) + 2.0 ** -19 * abs(float(y)) + 448 * 2.0 ** -149 + 2.0 ** -4 * abs(float(y))
        got = o.codes[:, 5].view(torch.float8_e4m3fn).double() * o.sf[:, 0].double()
        assert (got - float(y)).abs().max() <= err
