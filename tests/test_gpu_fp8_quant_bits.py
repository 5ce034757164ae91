"""Fp8Quant's codes and scales bit for bit: sf = amax / 448 and 1 / sf rounded to f32, the code the nearest E4M3 of the f32 product of
the value and 1 / sf.  In 64 bits all three are exact but for one rounding each (a quotient of f32 numbers rounded by 64 bits first
is the f32 quotient; products of two f32 numbers are exact), so nothing is left to a tolerance.  Widths that end inside a tile of 128
columns, rows that end inside one of 32, 64 and 128; the same bits in every call."""
import pytest
import torch

from fp8_ref import BF, DEV, F32, up_to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def tokens(T, H, dt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    v = r(T, H) * torch.exp2(3 * r(T, 1)) * torch.exp2(3 * r(1, H))
    v[T // 2] = 0
    return v.to(dt)


def definition(v, br, bc):
    R, C = v.shape
    pad = torch.nn.functional.pad(v.double(), (0, -C % bc, 0, -R % br))
    amax = pad.reshape(up_to(R, br), br, up_to(C, bc), bc).abs().amax((1, 3))
    sf = (amax / 448).float()
    inv = torch.where(sf > 0, 1 / sf.double(), torch.ones_like(amax)).float()
    each = inv.double().repeat_interleave(br, 0)[:R].repeat_interleave(bc, 1)[:, :C]
    return (v.double() * each).float().to(torch.float8_e4m3fn).view(torch.uint8), sf


def same(codes, sf, v, br, bc, what):
    q, s = definition(v, br, bc)
    assert torch.equal(sf, s), what + " scales"
    assert torch.equal(codes, q), f"{what}: {int((codes != q).sum())} of {q.numel()} codes"


@pytest.mark.parametrize("H", [16, 32, 48, 64, 80, 112, 128, 144, 176, 240, 272, 1040])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_widths(m, H, dt):
    op = m.Fp8Quant(H, dtype=dt, device=DEV)
    for T in (1, 3, 4, 5, 16, 17, 31, 64, 100, 128, 129, 1024, 1050, 3000):
        v = tokens(T, H, dt, T)
        for rows, cols in ((True, False), (False, True), (True, True)):
            for _ in range(2):
                o = op.forward(v, rows=rows, cols=cols)
                if rows:
                    same(o.codes, o.sf, v, 1, 128, f"{T} rows")
                if cols:
                    same(o.col_codes, o.col_sf, v, 128, 1, f"{T} columns")
        o = op.weights(v)
        same(o.codes, o.sf, v, 128, 128, f"{T} blocks")


def test_a_training_batch(m):
    """4096 x 7168, ten calls into buffers that hold other values before."""
    T, H = 4096, 7168
    op = m.Fp8Quant(H, device=DEV)
    out = op.buffers(T, cols=True)
    for seed in range(3):
        v = tokens(T, H, BF, seed)
        for _ in range(3):
            for t in (out.codes, out.sf, out.col_codes, out.col_sf):
                t.fill_(77)
            op.forward(v, cols=True, out=out)
            same(out.codes, out.sf, v, 1, 128, "rows")
            same(out.col_codes, out.col_sf, v, 128, 1, "columns")
