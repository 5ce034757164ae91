"""The last token counts below 2^31: a step past the last token does not fit
an int there.  Rows are as short as they can be (4 to 9 GB a tensor), and all
of them are checked.

Tolerance of the norm: one bf16 rounding of a value that f32 holds to a few
units, 2^-8."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
T = 2 ** 31 - 1
STEP = 1 << 28


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def pieces(T):
    return [slice(a, min(a + STEP, T)) for a in range(0, T, STEP)]


@pytest.mark.parametrize("T", [T, T - 31])
def test_router(m, T):
    x = torch.empty(T, 2, dtype=BF, device=DEV)
    for p in pieces(T):
        x[p].normal_(generator=torch.Generator(device=DEV).manual_seed(p.start % 997))
    op = m.Router(2, 1, balance_coef=1.0, logits_dtype=BF, max_tokens=T, device=DEV)
    out = op.forward_train(x)
    ones = 0
    for p in pieces(T):
        want = (x[p, 1] > x[p, 0]).int()                 # ties to the lower expert
        assert torch.equal(out.topk_idx[p, 0], want) and (out.topk_weights[p] == 1).all()
        ones += int(want.sum(dtype=torch.int64))
    assert out.counts.tolist() == [[T - ones, ones]] and out.tokens.tolist() == [T, 1, T]
    d = torch.full((T, 2), 5.0, dtype=BF, device=DEV)
    op.backward(x, out, d_weights=out.topk_weights, out=d)
    assert all((d[p] == 0).all() for p in pieces(T))     # a lone renormalised weight is 1 whatever the logits


def test_norm(m):
    x = torch.empty(T, 1, dtype=BF, device=DEV)
    for p in pieces(T):
        x[p].normal_(generator=torch.Generator(device=DEV).manual_seed(p.start % 997))
    out = m.BlockNorm(1, eps=0.5, device=DEV).forward(x, w_pre=torch.full((1,), 2.0, device=DEV))
    for p in pieces(T):
        v = x[p].float()
        r = (v * v + 0.5).rsqrt()
        assert torch.allclose(out.rstd_pre[p], r[:, 0], rtol=2.0 ** -20, atol=0)
        assert ((out.n[p].float() - 2 * v * r).abs() <= 2.0 ** -8 * (2 * v * r).abs()).all()
