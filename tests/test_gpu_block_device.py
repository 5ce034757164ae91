"""The library launches on the current device: a call of an operator that
lives on another one is refused before its tensors are looked at and before
anything reaches the library.  (The operators here are made to say that they
live on a second GPU; there need not be one.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def calls(m):
    """Name -> (operator, its call)"""
    x, w, l = torch.zeros(3, 256, dtype=BF, device=DEV), torch.ones(256, device=DEV), torch.zeros(3, 8, device=DEV)
    one, r1, x64 = torch.ones((), device=DEV), torch.ones(3, device=DEV), x[:, :64].contiguous()
    norm, route, lin = m.BlockNorm(256, device=DEV), m.Router(8, 2, max_tokens=4, device=DEV), m.Fp4Linear(64, 8, device=DEV)
    codes, sf = torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.zeros(8, 2, dtype=torch.uint8, device=DEV)
    lin.transform_weights(codes, sf)
    o, g, r, d, y = norm.buffers(3, block=False), norm.grad_buffers(3, block=False), route.buffers(3, 1), l.clone(), lin.buffers(3)
    fwd = route.forward_train(l)
    return {"norm": (norm, lambda s: norm.forward(x, w_pre=w, out=o, stream=s)),
            "norm backward": (norm, lambda s: norm.backward(x, dn=x, w_pre=w, rstd_pre=r1, out=g, stream=s)),
            "route": (route, lambda s: route.forward(l, out=r, stream=s)),
            "losses": (route, lambda s: route.forward_train(l, out=r, stream=s)),
            "given": (route, lambda s: route.balance_loss(l, r.topk_idx, out=r, stream=s)),
            "router backward": (route, lambda s: route.backward(l, fwd, d_loss=one, out=d, stream=s)),
            "transform": (lin, lambda s: lin.transform_weights(codes, sf, stream=s)),
            "linear": (lin, lambda s: lin.forward(x64, out=y, stream=s))}


@pytest.mark.parametrize("name", ["norm", "norm backward", "route", "losses", "given", "router backward", "transform", "linear"])
@pytest.mark.parametrize("side", [False, True], ids=["default", "side"])
def test_another_current_device_is_refused(m, monkeypatch, name, side):
    from moe_expert_ffn_gb300 import block
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    op, call = calls(m)[name]
    call(stream)
    torch.cuda.synchronize()
    monkeypatch.setattr(block, "_current_stream", lambda index: 0)
    monkeypatch.setattr(op, "_dev", 1)
    with pytest.raises(RuntimeError, match="cuda:1.*cuda:0"):
        call(stream)
