"""A router's weight so small that an expert's activations have scales whose reciprocal is past the f32 range, beside columns that are
zero: the token's output is the zero that such values round to, and not a NaN."""
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


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("T", [1, 4, 64, 700, 4096])
def test_no_nan(m, T, fmt):
    import moe_synth
    H, I, E, k = 256, 256, 4, 2
    wl = moe_synth.custom(T, H, I, E, k, wfmt=m.MOE_W_FP4_E2M1_UE8M0_32 if fmt == "fp4" else 0)
    i = moe_synth.make_inputs(wl, device="cpu")
    t = {n: v.to(DEV) for n, v in i.items()}
    w1 = t["w1"].clone()
    w1[:, 3::7] = 0                     # gate and up rows of zeros: activations that are zero
    layer = m.MoELayer(T, H, I, E, k, wfmt=wl.wfmt, device=DEV)
    layer.transform_weights(w1, t["w1_sf"], t["w2"], t["w2_sf"])
    plain = layer.forward(t["x"], t["x_sf"], t["topk_idx"], t["topk_weights"]).float()
    assert torch.isfinite(plain).all()
    for tiny in (1e-36, 1e-38, 1e-40, 1e-44):
        w = t["topk_weights"].clone()
        w[::2] = tiny                   # both slots of every other token
        w[1::4, 1] = tiny               # the second slot of some others
        y = layer.forward(t["x"], t["x_sf"], t["topk_idx"], w).float()
        assert torch.isfinite(y).all(), tiny
        assert y[::2].abs().max() <= 1e-30
    assert layer.device_status() == m.MOE_OK
