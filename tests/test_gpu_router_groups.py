"""Routing limited to groups of experts against the definition: which groups, which experts, ties, closed groups, close scores
(keys are the f32 next to the exact sigmoid, plus the bias in f32: choices have to be equal), every lane and register layout;
weights, losses and gradient as without groups for the same choice.

Tolerances are those of the ungrouped router (test_gpu_router.py): 2^-16 of a weight."""
import math

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


def make(T, E, dtype=F32, seed=0):
    return torch.randn(T, E, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def pick(v, k):
    val, idx = torch.sort(v, dim=1, descending=True, stable=True)
    return torch.where(val[:, :k] > -math.inf, idx[:, :k], -1)


def ref_choice(logits, bias, k, groups, use, kind, on_score):
    x = logits.float()
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x).clamp(max=torch.finfo(F32).max)
    key = torch.where(x > -math.inf, torch.sigmoid(x.double()).float(), x) if on_score else x
    if bias is not None:
        key = key + bias
    key = torch.where(key.isnan() | (x == -math.inf), torch.full_like(key, -math.inf), key)
    T, E = x.shape
    two = torch.sort(key.view(T, groups, E // groups), dim=2, descending=True).values
    score = two[:, :, 0]
    if kind == "top2" and E // groups > 1:
        score = score + torch.where(two[:, :, 1] > -math.inf, two[:, :, 1], torch.zeros_like(score))
    at = pick(score, use)
    on = torch.zeros(T, groups + 1, dtype=torch.bool, device=x.device).scatter_(1, torch.where(at < 0, groups, at), True)
    return pick(key.masked_fill(~on[:, :groups].repeat_interleave(E // groups, 1), -math.inf), k).to(torch.int32)


LAYOUTS = [(2, 1), (2, 8), (4, 8), (8, 8), (3, 5), (8, 4), (2, 32), (2, 16), (4, 9), (16, 4), (32, 1), (8, 32), (4, 64), (16, 16), (8, 20),
           (12, 40), (5, 29), (32, 32), (2, 512), (31, 31), (7, 100)]


@pytest.mark.parametrize("groups,size", LAYOUTS)
@pytest.mark.parametrize("kind", ["max", "top2"])
def test_choice(m, groups, size, kind):
    E = groups * size
    bias = 0.3 * torch.randn(E, generator=torch.Generator().manual_seed(1)).to(DEV)
    for use in sorted({1, max(1, groups // 2), groups - 1, groups}):
        for k in sorted({1, min(2, use * size), min(8, use * size), min(13, use * size), min(32, use * size)}):
            for score, on, b, dt in (("softmax", "logit", None, F32), ("softmax", "logit", bias, BF), ("sigmoid", "score", bias, F32),
                                     ("sigmoid", "score", None, F32), ("sigmoid", "logit", None, BF), ("sigmoid", "score", bias, BF)):
                T = 83
                x = make(T, E, dt, seed=use + k)
                x[7] = -math.inf
                x[8, :size] = -math.inf
                x[9, 1:] = -math.inf
                x[10, 0] = math.nan
                x[11, E - 1] = math.inf
                x[12] = 0.5                                          # all equal: ties to the lowest group and expert
                x[13] = x[13].mul(2).round()                         # many ties
                r = m.Router(E, k, score=score, logits_dtype=dt, bias_on=on, groups=groups, topk_groups=use, group_score=kind, device=DEV)
                o = r.forward(x, b)
                ref = ref_choice(x, b, k, groups, use, kind, on == "score" and (use < groups))
                if on == "score" and use == groups:
                    continue                                         # without a limit the scores are f32 ones (test_gpu_router_score_bias.py)
                assert torch.equal(o.topk_idx, ref), (use, k, score, on, dt)
                p = torch.softmax(x.double().clamp(max=3e38), 1) if score == "softmax" else torch.sigmoid(x.double())
                p[7] = 0
                w = torch.gather(p.nan_to_num(0), 1, ref.long().clamp(min=0)) * (ref >= 0)
                w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
                rows = [t for t in range(T) if t not in (10, 11)]
                assert ((o.topk_weights.double() - w).abs() <= 2.0 ** -16 * w)[rows].all()


@pytest.mark.parametrize("kind", ["max", "top2"])
@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_close_scores(m, kind, dt):
    """Keys that only exact sigmoids order: logits a few units in the last place apart, biases that bring different scores
    together, saturated scores."""
    T, E, groups, use, k = 4000, 256, 8, 4, 8
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, E, generator=g)
    near = x[:, :1].clone()
    x[:1000, ::3] = near[:1000] * (1 + torch.randint(-3, 4, (1000, 86), generator=g) * 2.0 ** -23)
    x[1000:2000] = x[1000:2000].mul(2).round() / 2
    x[2000:3000] += 9                                            # 1 - sigmoid of 2^-13 and less
    x[3000:] -= 12
    bias = torch.zeros(E)
    bias[::5] = torch.sigmoid(torch.tensor(0.5)) - torch.sigmoid(torch.tensor(1.0))     # 1.0 with it is close to 0.5 without
    x, bias = x.to(dt).to(DEV), bias.to(DEV)
    r = m.Router(E, k, score="sigmoid", logits_dtype=dt, bias_on="score", groups=groups, topk_groups=use, group_score=kind, device=DEV)
    for b in (bias, None):
        assert torch.equal(r.forward(x, b).topk_idx, ref_choice(x, b, k, groups, use, kind, True))


def test_many_tokens_and_pitches(m):
    T, E = 30001, 256
    x = make(T, E, F32, 5)
    wide = torch.full((T, E + 3), math.nan, device=DEV)
    wide[:, 1:E + 1] = x
    bias = 0.1 * make(1, E, F32, 6)[0]
    r = m.Router(E, 8, score="sigmoid", bias_on="score", groups=8, topk_groups=4, group_score="top2", device=DEV)
    ref = ref_choice(x, bias, 8, 8, 4, "top2", True)
    a, b = r.forward(x, bias), r.forward(wide[:, 1:E + 1], bias)
    assert torch.equal(a.topk_idx, ref) and torch.equal(b.topk_idx, ref) and torch.equal(a.topk_weights, b.topk_weights)


@pytest.mark.parametrize("groups,size,score,dt", [(8, 32, "sigmoid", F32), (4, 64, "softmax", BF), (8, 8, "sigmoid", BF), (5, 29, "softmax", F32),
                                                  (12, 40, "sigmoid", F32), (3, 5, "softmax", F32)])
def test_losses_and_gradient_are_those_of_the_choice(m, groups, size, score, dt):
    """Bit for bit what the ungrouped router gives for this choice: counts and means of its losses, its gradient."""
    E, k, T = groups * size, 4, 700
    x = make(T, E, dt, 3)
    x[5] = -math.inf
    off = torch.tensor([0, 100, 100, 650, T], dtype=torch.int32, device=DEV)
    kw = dict(score=score, balance_coef=0.1, z_coef=0.01 if score == "softmax" else 0.0, logits_dtype=dt, max_tokens=T, max_seqs=4, device=DEV)
    grouped = m.Router(E, k, groups=groups, topk_groups=2, group_score="top2", **kw)
    plain = m.Router(E, k, **kw)
    o = grouped.forward_train(x, seq_offsets=off)
    assert torch.equal(o.topk_idx, grouped.forward(x).topk_idx) and torch.equal(o.topk_weights, grouped.forward(x).topk_weights)
    assert torch.equal(o.topk_idx, ref_choice(x, None, k, groups, 2, "top2", False))
    given = plain.balance_loss(x, o.topk_idx, off)
    assert torch.equal(o.counts, given.counts) and torch.equal(o.seq_tokens, given.seq_tokens)
    assert (o.loss - given.loss).abs().max() <= 2.0 ** -16 * given.loss.abs().max()
    assert (o.prob_mean - given.prob_mean).abs().max() <= 2.0 ** -16 * given.prob_mean.max()
    dw = make(T, k, F32, 9)
    one = torch.ones((), device=DEV)
    a = grouped.backward(x, o, d_weights=dw, d_loss=one)
    given.topk_idx = o.topk_idx
    b = plain.backward(x, given, d_weights=dw, d_loss=one)
    assert torch.equal(a, b)


def test_gradient_against_differences(m):
    """Through the weights of a fixed choice, in 64 bits around f32 logits."""
    E, k, T, groups = 24, 3, 20, 4
    x = make(T, E, F32, 8)
    r = m.Router(E, k, score="sigmoid", groups=groups, topk_groups=2, bias_on="score", device=DEV)
    o = r.forward(x)
    dw = make(T, k, F32, 2)
    d = r.backward(x, o, d_weights=dw).double()
    idx, X, h = o.topk_idx.long(), x.double(), 1e-6

    def value(z):
        w = torch.gather(torch.sigmoid(z), 1, idx)
        return (w / w.sum(1, keepdim=True) * dw).sum(1)

    for e in range(E):
        step = torch.zeros_like(X)
        step[:, e] = h
        diff = (value(X + step) - value(X - step)) / (2 * h)
        assert (diff - d[:, e]).abs().max() <= 1e-5


def test_repeats_and_capture(m):
    T, E = 1000, 256
    x, bias = make(T, E, F32, 1), 0.1 * make(1, E, F32, 2)[0]
    r = m.Router(E, 8, score="sigmoid", bias_on="score", groups=8, topk_groups=4, group_score="top2", balance_coef=0.1, max_tokens=T, device=DEV)
    a = r.forward_train(x, bias)
    out = r.buffers(T, num_seqs=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        r.forward_train(x, bias, out=out)
        with torch.cuda.graph(g, stream=s):
            r.forward_train(x, bias, out=out)
    out.topk_idx.zero_()
    g.replay()
    torch.cuda.synchronize()
    for n in ("topk_idx", "topk_weights", "loss", "counts", "prob_mean"):
        assert torch.equal(getattr(a, n), getattr(out, n))


def test_no_tokens(m):
    r = m.Router(64, 4, groups=8, topk_groups=2, balance_coef=0.1, max_tokens=4, device=DEV)
    assert r.forward(torch.empty(0, 64, device=DEV)).topk_idx.shape == (0, 4)
    assert (r.forward_train(torch.empty(0, 64, device=DEV)).loss == 0).all()
