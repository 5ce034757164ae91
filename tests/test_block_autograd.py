"""The block operators take no part in autograd, and a forward call says so
when its inputs require gradients.  (On CPU tensors nothing is launched, which
is the error that every call here ends in.)"""
import warnings

import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def calls(m, wants):
    x, w, l = torch.zeros(3, 256, dtype=BF), torch.ones(256), torch.zeros(3, 8)
    few = torch.zeros(3, 64, dtype=BF)
    for t in {"x": (x, few), "w": (w,), "l": (l,)}.get(wants, ()):
        t.requires_grad_()
    norm, route, lin = m.BlockNorm(256, device="cpu"), m.Router(8, 2, max_tokens=4, device="cpu"), m.Fp4Linear(64, 8, device="cpu")
    lin._ready = True
    idx = torch.zeros(3, 2, dtype=torch.int32)
    return {"norm x": lambda: norm.forward(x, w_pre=w), "norm w": lambda: norm.forward(x, w_pre=w),
            "route l": lambda: route.forward(l), "losses l": lambda: route.forward_train(l), "given l": lambda: route.balance_loss(l, idx),
            "linear x": lambda: lin.forward(few)}


@pytest.mark.parametrize("name", ["norm x", "norm w", "route l", "losses l", "given l", "linear x"])
def test_inputs_with_a_graph(m, name):
    call = calls(m, name.split()[1])[name]
    with pytest.warns(UserWarning, match="no part in autograd"):
        with pytest.raises(RuntimeError, match="CPU"):
            call()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning):                 # a warning made an error is raised as one
            call()
        with torch.no_grad(), pytest.raises(RuntimeError, match="CPU"):
            call()
        with pytest.raises(RuntimeError, match="CPU"):
            calls(m, None)[name]()


def test_backward_passes_are_for_that(m):
    x, w = torch.zeros(3, 256, dtype=BF, requires_grad=True), torch.ones(256, requires_grad=True)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(RuntimeError, match="CPU"):
            m.BlockNorm(256, device="cpu").backward(x, dn=x, w_pre=w, rstd_pre=torch.ones(3))
