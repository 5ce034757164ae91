"""Losses and gradients of a choice made elsewhere: what balance_loss returns
goes into backward as it is.

Tolerance as in the router's tests: gradients are sums of terms of either
sign, each a quotient of f32 exponentials: 2^-16 of the sum of their
magnitudes."""
import math

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


def given(T, E, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].int()
    return x, idx, torch.randn(T, k, generator=g)


def weight_grad(x, idx, dw, scale=1.0):
    """Gradient through renormalised softmax weights and the magnitude of its terms, in 64 bits."""
    x, dw, idx = x.double(), scale * dw.double(), idx.long()
    w = torch.softmax(torch.gather(x, 1, idx), 1)
    dot = (w * dw).sum(1, keepdim=True)
    z = torch.zeros_like(x)
    return z.scatter(1, idx, w * (dw - dot)), z.scatter(1, idx, w * (dw.abs() + (w * dw).abs().sum(1, keepdim=True)))


def close(got, ref, mag):
    assert ((got.double().cpu() - ref).abs() <= 2.0 ** -16 * mag + 1e-30).all()


@pytest.mark.parametrize("own_buffers", [False, True])
@pytest.mark.parametrize("E,k", [(16, 3), (256, 8)])
def test_result_goes_into_backward(m, E, k, own_buffers):
    T = 75
    x, idx, dw = given(T, E, k)
    op = m.Router(E, k, balance_coef=1.0, weight_scale=1.5, max_tokens=T, device=DEV)
    buf = op.buffers(T, 1) if own_buffers else None
    if own_buffers:
        buf.topk_idx.fill_(0)                            # what it holds is no choice of anybody's
    gi = idx.to(DEV)
    out = op.balance_loss(x.to(DEV), gi, out=buf)
    assert torch.equal(out.topk_idx, gi)
    d = op.backward(x.to(DEV), out, d_weights=dw.to(DEV))
    close(d, *weight_grad(x, idx, dw, 1.5))
    if own_buffers:                                      # the buffers are still the caller's, and the choice its own
        assert out.loss is buf.loss and out.counts is buf.counts and (buf.topk_idx == 0).all()
        op.forward_train(x.to(DEV), out=buf)
        assert torch.equal(gi.cpu(), idx)


def test_no_weights_that_nobody_wrote(m):
    x, idx, _ = given(9, 8, 2)
    out = m.Router(8, 2, balance_coef=1.0, max_tokens=9, device=DEV).balance_loss(x.to(DEV), idx.to(DEV))
    assert out.topk_weights is None
