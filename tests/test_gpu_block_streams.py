"""What a call allocates for a stream of its own belongs to that stream: the
memory goes back to it, and to nobody who works on another one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
T, H = 1531, 2048


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def owner(t):
    """The stream whose memory t lies in."""
    return next(g["stream"] for g in torch.cuda.memory_snapshot() if 0 <= t.data_ptr() - g["address"] < g["total_size"])


def calls(m):
    x, w = torch.randn(T, H, device=DEV).to(BF), torch.ones(H, device=DEV)
    norm, route = m.BlockNorm(H, device=DEV), m.Router(256, 8, balance_coef=1.0, max_tokens=T, device=DEV)
    logits = torch.randn(T, 256, device=DEV)
    rstd = norm.forward(x, w_pre=w).rstd_pre
    fwd, one = route.forward_train(logits), torch.ones((), device=DEV)
    lin = m.Fp4Linear(64, 40000, device=DEV)
    lin.transform_weights(torch.zeros(40000, 32, dtype=torch.uint8, device=DEV), torch.zeros(40000, 2, dtype=torch.uint8, device=DEV))
    few = x[:16, :64].contiguous()
    torch.cuda.synchronize()
    return {"norm": lambda s: norm.forward(x, w_pre=w, stream=s).n,
            "norm backward": lambda s: norm.backward(x, dn=x, w_pre=w, rstd_pre=rstd, stream=s).dresidual,
            "route": lambda s: route.forward(logits, stream=s).topk_idx,
            "losses": lambda s: route.forward_train(logits, stream=s).topk_weights,
            "given": lambda s: route.balance_loss(logits, fwd.topk_idx, stream=s).prob_mean,
            "router backward": lambda s: route.backward(logits, fwd, d_loss=one, stream=s),
            "linear": lambda s: lin.forward(few, stream=s)}


@pytest.mark.parametrize("name", ["norm", "norm backward", "route", "losses", "given", "router backward", "linear"])
def test_outputs_belong_to_the_stream(m, name):
    call, s = calls(m)[name], torch.cuda.Stream()
    torch.cuda.synchronize()
    here = call(None)
    s.wait_stream(torch.cuda.current_stream())
    out = call(s)
    torch.cuda.synchronize()
    assert torch.equal(out, here)
    assert owner(out) == s.cuda_stream and owner(here) == torch.cuda.current_stream().cuda_stream
