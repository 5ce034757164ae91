"""Choices by sigmoid score + bias against the definition in 64 bits.

Tolerance.  The score is right to 2^-19 of itself or 2^-40 (its exponential's
argument is rounded once: 2^-24 of 1.44 |l|; the rest are a few units), and
the sum is rounded to f32: two keys further apart than both their errors have
to come out in order, whichever of nearer ones is taken."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def keys(x, bias):
    """64-bit keys and their errors' bounds (-inf: closed)"""
    x, bias = x.double().cpu(), bias.double().cpu()
    s = torch.sigmoid(torch.where(torch.isnan(x), -math.inf, x))
    key = s + bias
    key = torch.where(torch.isnan(key) | torch.isnan(x) | (x == -math.inf), -math.inf, key)
    return key, 2.0 ** -19 * s + 2.0 ** -40 + 2.0 ** -24 * torch.nan_to_num(key, 0, 0, 0).abs()


def check_choice(idx, x, bias, k):
    key, err = keys(x, bias)
    idx = idx.cpu().long()
    T, E = key.shape
    open_ = (key > -math.inf).sum(1)
    slot = torch.arange(k)
    assert torch.equal(idx >= 0, slot[None] < open_[:, None])
    on = idx >= 0
    c = idx.clamp_min(0)
    kc, ec = key.gather(1, c), err.gather(1, c)
    assert (kc[on] > -math.inf).all()
    seen = torch.zeros(T, E, dtype=torch.int64).scatter_add(1, c, on.long())
    assert seen.max() <= 1
    pair = on[:, 1:] & torch.isfinite(kc[:, 1:])
    assert (kc[:, :-1] - kc[:, 1:] >= -(ec[:, :-1] + ec[:, 1:]))[pair].all()
    rest = torch.where(seen > 0, -math.inf, key - err).amax(1)
    low = torch.where(on, kc + ec, math.inf).amin(1)
    assert (low >= rest).all()                           # no key left out is above a chosen one by more than their errors
    return c, on


EXPERTS = [(2, 1), (8, 2), (33, 8), (64, 6), (128, 6), (256, 8), (300, 12), (512, 20), (1024, 32)]


@pytest.mark.parametrize("E,k", EXPERTS)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
def test_choice_weights_and_counts(m, E, k, dtype, renorm):
    T = 203
    g = torch.Generator().manual_seed(E + k)
    x = (2.0 * torch.randn(T, E, generator=g)).to(dtype)
    x[5] = -math.inf                                     # a padding token
    x[6, ::2] = math.nan
    x[7, 0] = math.inf
    x[8, : E - 1] = -math.inf
    bias = 0.3 * torch.randn(E, generator=g)
    bias[E // 2] = -math.inf                             # taken out for everybody
    x, bias = x.to(DEV), bias.to(DEV)
    op = m.Router(E, k, score="sigmoid", renormalize=renorm, weight_scale=2.5, logits_dtype=dtype, balance_coef=1.0, max_tokens=T,
                  bias_on="score", device=DEV)
    out = op.forward(x, bias)
    c, on = check_choice(out.topk_idx, x, bias, k)
    s = torch.where(on, torch.sigmoid(x.double().cpu()).gather(1, c), 0.0)
    w = 2.5 * (s / s.sum(1, keepdim=True).clamp_min(1e-300) if renorm else s)
    assert ((out.topk_weights.double().cpu() - w).abs() <= 2.0 ** -16 * w).all()
    train = op.forward_train(x, bias)
    assert torch.equal(train.topk_idx, out.topk_idx) and torch.equal(train.topk_weights, out.topk_weights)
    real = (torch.nan_to_num(x.float(), -math.inf) > -math.inf).any(1).cpu()
    assert np.array_equal(train.counts.cpu().numpy()[0], np.bincount(c[on & real[:, None]].numpy(), minlength=E))
    # without a bias the scores' order is the logits'
    plain = m.Router(E, k, score="sigmoid", logits_dtype=dtype, device=DEV).forward(x)
    assert torch.equal(op.forward(x).topk_idx, plain.topk_idx)


def test_it_differs_from_a_bias_on_the_logits(m):
    x, bias = torch.tensor([[4.0, 0.0]], device=DEV), torch.tensor([0.0, 0.6], device=DEV)
    got = {on: m.Router(2, 1, score="sigmoid", bias_on=on, device=DEV).forward(x, bias).topk_idx.item() for on in ("logit", "score")}
    assert got == {"logit": 0, "score": 1}
    assert m.Router(2, 1, score="sigmoid", device=DEV).forward(x, bias).topk_idx.item() == 0


@pytest.mark.parametrize("E,k", [(16, 4), (256, 8), (1000, 12)])
def test_ties_go_to_the_lowest_expert(m, E, k):
    """Scores that are all 1, or all equal, leave the biases to decide, and equal biases the numbers."""
    x = torch.stack([torch.linspace(30.0, 90.0, E), torch.full((E,), -0.7)]).to(DEV)
    op = m.Router(E, k, score="sigmoid", bias_on="score", device=DEV)
    assert op.forward(x, torch.zeros(E, device=DEV)).topk_idx.cpu().tolist() == [list(range(k))] * 2
    bias = torch.zeros(E, device=DEV)
    bias[E - 3:] = 0.25
    want = [E - 3, E - 2, E - 1] + list(range(k - 3))
    assert op.forward(x, bias).topk_idx.cpu().tolist() == [want] * 2


@pytest.mark.parametrize("E,k", [(256, 8), (512, 12)])
def test_many_tokens(m, E, k):
    """Small spreads, where choices hang on the keys' last bits."""
    T = 20000
    g = torch.Generator().manual_seed(E)
    x, bias = (0.01 * torch.randn(T, E, generator=g)).to(DEV), (0.01 * torch.randn(E, generator=g)).to(DEV)
    check_choice(m.Router(E, k, score="sigmoid", bias_on="score", device=DEV).forward(x, bias).topk_idx, x, bias, k)
