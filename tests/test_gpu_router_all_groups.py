"""Routing whose groups are all taken: by scores the keys are those of any other grouped call, the f32 next to the exact sigmoid plus the
bias in f32, so the choice is that of a stable sort of them; by logits it is the router's without groups."""
import math

import pytest
import torch

from test_gpu_router_groups import BF, DEV, F32, m, make, ref_choice  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,size", [(2, 1), (4, 8), (8, 8), (3, 5), (4, 64), (8, 32), (16, 16), (12, 40), (31, 31), (32, 32)])
@pytest.mark.parametrize("kind", ["max", "top2"])
@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_by_scores(m, groups, size, kind, dt):  # noqa: F811
    E, T = groups * size, 300
    bias = 0.3 * torch.randn(E, generator=torch.Generator().manual_seed(1)).to(DEV)
    x = make(T, E, dt, 7)
    x[100:200] += 20                                # saturated: the scores are 1, the logits differ
    x[200:250] *= 12
    x[3] = -math.inf
    x[4, 1:] = -math.inf
    x[5] = 30.0
    x[5, 0] = 20.0
    x[6, E - 1] = math.inf
    x[7, 0] = math.nan
    for k in sorted({1, min(8, E), min(13, E), min(32, E)}):
        r = m.Router(E, k, score="sigmoid", logits_dtype=dt, bias_on="score", groups=groups, topk_groups=groups, group_score=kind, device=DEV)
        for b in (bias, None):
            assert torch.equal(r.forward(x, b).topk_idx, ref_choice(x, b, k, groups, groups, kind, True)), (k, b is None)


def test_saturated_scores_tie(m):  # noqa: F811
    """Logits 20 and 30 have the score 1 both: the lower expert comes first, in the call with a limit and in that without."""
    x = torch.full((1, 8), -5.0, device=DEV)
    x[0, 1], x[0, 2] = 20.0, 30.0
    for use in (3, 4):
        r = m.Router(8, 2, score="sigmoid", bias_on="score", groups=4, topk_groups=use, device=DEV)
        assert r.forward(x).topk_idx.tolist() == [[1, 2]], use


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_losses_and_gradient(m, dt):  # noqa: F811
    """By scores with a bias: the losses are those of the choice, and the gradient, as the ungrouped router gives them for it."""
    E, k, T = 64, 4, 700
    x, bias = make(T, E, dt, 3), 0.2 * make(1, E, F32, 4)[0]
    off = torch.tensor([0, 100, 100, 650, T], dtype=torch.int32, device=DEV)
    kw = dict(score="sigmoid", bias_on="score", balance_coef=0.1, logits_dtype=dt, max_tokens=T, max_seqs=4, device=DEV)
    all_of, plain = m.Router(E, k, groups=8, topk_groups=8, **kw), m.Router(E, k, **kw)
    o = all_of.forward_train(x, bias, seq_offsets=off)
    assert torch.equal(o.topk_idx, ref_choice(x, bias, k, 8, 8, "max", True))
    given = plain.balance_loss(x, o.topk_idx, off)
    assert torch.equal(o.counts, given.counts) and torch.equal(o.seq_tokens, given.seq_tokens)
    assert (o.loss - given.loss).abs().max() <= 2.0 ** -16 * given.loss.abs().max()
    dw, one = make(T, k, F32, 9), torch.ones((), device=DEV)
    a = all_of.backward(x, o, d_weights=dw, d_loss=one)
    given.topk_idx = o.topk_idx
    assert torch.equal(a, plain.backward(x, given, d_weights=dw, d_loss=one))


@pytest.mark.parametrize("score,on,dt", [("softmax", "logit", F32), ("softmax", "logit", BF), ("sigmoid", "logit", F32)])
def test_by_logits(m, score, on, dt):  # noqa: F811
    E, T, k = 256, 500, 8
    x, bias = make(T, E, dt, 5), 0.3 * make(1, E, F32, 6)[0]
    x[3], x[4, 9], x[5, 8], x[6] = -math.inf, math.inf, math.nan, 0.5
    kw = dict(score=score, bias_on=on, logits_dtype=dt, device=DEV)
    for b in (bias, None):
        a, p = (m.Router(E, k, **g, **kw).forward(x, b) for g in (dict(groups=8, topk_groups=8), {}))
        assert torch.equal(a.topk_idx, p.topk_idx) and torch.equal(a.topk_weights, p.topk_weights)
