"""FP8 products of many 256 x 256 tiles, several to each pair of CTAs: outputs and added inputs share the operands' stages, few and many
blocks to a tile, ends inside tiles; SwiGLU with an added input in every kernel.  Tolerances: fp8_ref.py; an added input enters the sum of
magnitudes' last rounding, 2^-23 of both."""
import math

import pytest
import torch

from fp8_ref import BF, DEV, F32, close, close_codes, product, random_codes, swiglu, up, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    yield mod
    assert mod.lib().moe_fp8_linear_status() == mod.MOE_OK


def noise(R, C, dt, seed):
    return torch.randn(R, C, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dt)


def with_add(y, err, add):
    return y + add.double(), err + 2.0 ** -23 * (y.abs() + add.abs().double())


# one to nine blocks; 4.7, 3.9 and 3.4 tiles a pair
@pytest.mark.parametrize("T,N,K", [(5000, 4624, 16), (4609, 4112, 144), (5000, 3344, 272), (4609, 4112, 400), (4400, 4112, 1040)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_forward(m, T, N, K, dt):
    x, x_sf = random_codes(T, K, 1, 128, 1)
    w, w_sf = random_codes(N, K, 128, 128, 2, scale=1 / K)
    y, err = product(values(x, x_sf, 1, 128), values(w, w_sf, 128, 128), up(K))
    op = m.Fp8Linear(K, N, out_dtype=dt, device=DEV)
    first = op.forward(x, x_sf, w, w_sf)
    close(first, y, err)
    assert torch.equal(op.forward(x, x_sf, w, w_sf), first)
    add = noise(T, N, dt, 3)
    both = with_add(y, err, add)
    close(op.forward(x, x_sf, w, w_sf, add=add), *both, "added")
    op.forward(x, x_sf, w, w_sf, add=add, out=add)
    close(add, *both, "in place")


@pytest.mark.parametrize("T,N,K", [(16, 4624, 4624), (144, 4112, 4112), (300, 4112, 3344), (520, 3344, 4112), (1100, 4112, 4112)])
def test_weight_gradient(m, T, N, K):
    dy, dy_sf = random_codes(T, N, 128, 1, 1)
    x, x_sf = random_codes(T, K, 128, 1, 2)
    dw, err = product(values(dy, dy_sf, 128, 1).t(), values(x, x_sf, 128, 1).t(), up(T))
    op = m.Fp8Linear(K, N, device=DEV)
    close(op.backward_weight(dy, dy_sf, x, x_sf), dw, err)
    add = noise(N, K, F32, 3)
    both = with_add(dw, err, add)
    op.backward_weight(dy, dy_sf, x, x_sf, add=add, out=add)
    close(add, *both, "in place")
    op.backward_weight(dy, dy_sf, x, x_sf, add=add, out=add)      # once more on top
    close(add, both[0] + dw, both[1] + err + 2.0 ** -22 * (both[0].abs() + dw.abs()), "twice")


@pytest.mark.parametrize("T,N,K", [(4609, 400, 4112), (5000, 272, 3344), (4609, 16, 4624)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_input_gradient(m, T, N, K, dt):
    dy, dy_sf = random_codes(T, N, 1, 128, 1)
    w, w_sf = random_codes(N, K, 128, 128, 2, scale=1 / N)
    dx, err = product(values(dy, dy_sf, 1, 128), values(w, w_sf, 128, 128).t(), up(N))
    add = noise(T, K, dt, 3)
    op = m.Fp8Linear(K, N, out_dtype=dt, device=DEV)
    close(op.backward_input(dy, dy_sf, w, w_sf), dx, err)
    close(op.backward_input(dy, dy_sf, w, w_sf, add=add), *with_add(dx, err, add), "added")


@pytest.mark.parametrize("T,N,K", [(1, 512, 272), (16, 256, 400), (40, 512, 144), (65, 768, 272), (300, 512, 400), (4609, 4096, 16), (5000, 3584, 272),
                                   (4400, 4096, 400)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_swiglu_with_an_added_input(m, T, N, K, dt):
    x, x_sf = random_codes(T, K, 1, 128, 1)
    w, w_sf = random_codes(N, K, 128, 128, 2, scale=1 / K)
    y, err = swiglu(*product(values(x, x_sf, 1, 128), values(w, w_sf, 128, 128), up(K)))
    add = noise(T, N // 2, dt, 3)
    op = m.Fp8Linear(K, N, act="swiglu", out_dtype=dt, device=DEV)
    close(op.forward(x, x_sf, w, w_sf), y, err)
    both = with_add(y, err, add)
    close(op.forward(x, x_sf, w, w_sf, add=add), *both, "added")
    op.forward(x, x_sf, w, w_sf, add=add, out=add)
    close(add, *both, "in place")
    o = m.Fp8Linear(K, N, act="swiglu", quant="fp8", act_clamp=math.inf, device=DEV).forward(x, x_sf, w, w_sf)
    close_codes(o.codes, o.sf, y, err, 1, 128)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_pitches_and_what_lies_around(m, dt):
    T, N, K = 4609, 4112, 144
    x, x_sf = random_codes(T, K, 1, 128, 1)
    w, w_sf = random_codes(N, K, 128, 128, 2, scale=1 / K)
    op = m.Fp8Linear(K, N, out_dtype=dt, device=DEV)
    add = noise(T, N, dt, 3)
    ref = op.forward(x, x_sf, w, w_sf, add=add)
    es = 16 // add.element_size()
    for pad, offset in ((es, 0), (3 * es, 2 * es)):
        yb = torch.full((T * (N + pad) + offset,), 5.0, dtype=dt, device=DEV)
        yv, ab = torch.as_strided(yb, (T, N), (N + pad, 1), offset), torch.full_like(yb, math.nan)
        av = torch.as_strided(ab, (T, N), (N + pad, 1), offset)
        av.copy_(add)
        op.forward(x, x_sf, w, w_sf, add=av, out=yv)
        assert torch.equal(yv, ref)
        keep = torch.ones_like(yb, dtype=torch.bool)
        torch.as_strided(keep, (T, N), (N + pad, 1), offset).fill_(False)
        assert (yb[keep] == 5.0).all()
