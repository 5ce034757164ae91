"""Gradients at slots whose expert is closed: a choice made elsewhere may name
an expert whose logit is -inf or NaN.  Its weight is 0 whatever the logits
are, so whatever gradient the caller holds for that slot, infinities and NaN
among them, reaches no logit.

Tolerance as in the router's tests: 2^-16 of the terms' magnitudes."""
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


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("E", [12, 200])
@pytest.mark.parametrize("held", [math.nan, math.inf, -math.inf, 3.0])
def test_closed_slot_gradient_is_ignored(m, E, score, renorm, held):
    T, k = 24, 3
    g = torch.Generator().manual_seed(E)
    x = torch.randn(T, E, generator=g)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].int()
    dw = torch.randn(T, k, generator=g)
    rows = torch.arange(T)
    x[rows, idx[rows, rows % k].long()] = torch.where(rows % 2 == 0, -math.inf, math.nan)
    dw[rows, rows % k] = held
    op = m.Router(E, k, score=score, renormalize=renorm, device=DEV)
    out = op.buffers(T)
    out.topk_idx = idx.to(DEV)
    d = op.backward(x.to(DEV), out, d_weights=dw.to(DEV)).double().cpu()
    # the definition in 64 bits, closed experts left out
    closed = torch.isnan(x) | torch.isinf(x)
    l = x.double().masked_fill(closed, -math.inf)
    sig = torch.sigmoid(l)
    s, slope = (torch.softmax(l, 1), 1.0) if score == "softmax" else (sig, 1 - sig)
    on = torch.zeros(T, E, dtype=torch.bool).scatter(1, idx.long(), True) & ~closed
    sel = torch.where(on, s, 0.0)
    w = sel / sel.sum(1, keepdim=True) if renorm else sel
    G = torch.zeros(T, E, dtype=torch.float64).scatter(1, idx.long(), torch.nan_to_num(dw.double(), 0.0, 0.0, 0.0)).masked_fill(closed, 0.0)
    dot = (w * G).sum(1, keepdim=True) if renorm or score == "softmax" else 0.0
    base = w if renorm else s
    ref = base * slope * (G - dot)
    mag = base * (G.abs() + (w * G).abs().sum(1, keepdim=True))
    assert torch.isfinite(d).all()
    assert ((d - ref).abs() <= 2.0 ** -16 * mag + 1e-30).all()
