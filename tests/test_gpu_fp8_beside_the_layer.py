"""Chains of FP8 linear calls of few and of many rows on two streams, the expert layer on a third: all of them take tensor memory, and
none may hold it while it waits for a kernel that still wants some.  Results are those of calls alone."""
import pytest
import torch

from fp8_ref import DEV, random_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


@pytest.mark.parametrize("rows", [(1, 16), (1, 40), (16, 600)])
def test_three_streams(m, rows):
    import moe_synth
    N, K = 2048, 2048
    op = m.Fp8Linear(K, N, device=DEV)
    w = random_codes(N, K, 128, 128, 2, scale=1 / K)
    x = [random_codes(T, K, 1, 128, T) for T in rows]
    alone = [op.forward(*a, *w) for a in x]
    out = [[op.buffers(T) for _ in range(60)] for T in rows]
    wl = moe_synth.custom(64, 512, 256, 8, 2)
    i = moe_synth.make_inputs(wl, device="cpu")
    layer = m.MoELayer(64, 512, 256, 8, 2, device=DEV)
    layer.transform_weights(*(i[n].to(DEV) for n in ("w1", "w1_sf", "w2", "w2_sf")))
    tokens = [i[n].to(DEV) for n in ("x", "x_sf", "topk_idx", "topk_weights")]
    y = layer.forward(*tokens).clone()
    ys = [torch.empty_like(y) for _ in range(30)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for n in range(60):
        for s, a, o in zip(streams, x, out):
            op.forward(*a, *w, out=o[n], stream=s)
        if n % 2:
            layer.forward(*tokens, y=ys[n // 2], stream=streams[2])
    torch.cuda.synchronize()
    assert op.device_status() == m.MOE_OK and layer.device_status() == m.MOE_OK
    for a, o in zip(alone, out):
        assert all(torch.equal(t, a) for t in o)
    assert all(torch.equal(t, y) for t in ys)
