"""Router against the definitions in 64 bits: choices (ties, closed experts,
masked rows, bias), weights, losses over ragged sequences, counts, and the
gradient of the logits against the formula and against differences.

Tolerances.  Choices and counts are whole numbers and have to be equal: keys
are f32 sums, compared exactly.  Weights and probabilities are quotients of
f32 exponentials: an exponential's error is 2 units plus that of its argument,
|l - m| 2^-24 (|l - m| < 100 where it matters), so 2^-16 relative is wide and
wrong terms are far outside it.  Losses and means are sums of such terms of
one sign: the same.  Gradients are sums of terms of either sign: 2^-16 of the
sum of their magnitudes, and one rounding (2^-8) in bf16.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
FLT_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def make(T, E, dtype=F32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(T, E, generator=g)).to(dtype).to(DEV)


def open_logits(logits):
    x = logits.float().cpu().numpy().astype(np.float64)
    x[np.isnan(x)] = -np.inf
    return np.minimum(x, FLT_MAX)


def ref_choice(logits, bias, k):
    x = open_logits(logits).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        key = x if bias is None else (x + bias.cpu().numpy()).astype(np.float32)
    key = np.where(np.isnan(key) | np.isneginf(x), -np.inf, key)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    return np.where(np.isneginf(np.take_along_axis(key, idx, 1)), -1, idx).astype(np.int32)


def ref_all(logits, idx, score, renorm, scale, k, offsets=None, alpha=0.0, beta=0.0, dw=None, d_loss=None):
    """Everything in 64 bits, token by token."""
    x = open_logits(logits)
    T, E = x.shape
    real = np.isfinite(x).any(1)
    m = np.where(real, x.max(1, initial=-np.inf), 0.0)
    with np.errstate(over="ignore"):
        ex = np.where(np.isfinite(x), np.exp(x - m[:, None]), 0.0)
        soft = ex / np.maximum(ex.sum(1, keepdims=True), 1e-300)
        lse = np.where(real, m + np.log(np.maximum(ex.sum(1), 1e-300)), 0.0)
        sig = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    sig = np.where(np.isfinite(x), sig, 0.0)
    s = soft if score == "softmax" else sig
    share = s / np.maximum(s.sum(1, keepdims=True), 1e-320)
    slope = 1 - sig if score == "sigmoid" else np.ones_like(x)
    hit = np.zeros((T, E))
    for j in range(idx.shape[1]):
        on = (idx[:, j] >= 0) & (idx[:, j] < E)
        hit[np.nonzero(on)[0], idx[on, j]] = 1
    sel = s * hit
    tot = sel.sum(1, keepdims=True)
    q = np.divide(sel, tot, out=np.zeros_like(sel), where=tot > 0) if renorm else sel
    o = {"weights": scale * np.take_along_axis(q, np.clip(idx, 0, E - 1), 1) * ((idx >= 0) & (idx < E))}
    g, gmag = np.zeros_like(x), np.zeros_like(x)
    off = [0, T] if offsets is None else list(offsets)
    S = len(off) - 1
    o["counts"], o["prob"], o["n"] = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    for i in range(S):
        r = slice(off[i], off[i + 1])
        o["n"][i] = real[r].sum()
        o["counts"][i] = (hit[r] * real[r, None]).sum(0)
        if o["n"][i]:
            o["prob"][i] = (share[r] * real[r, None]).sum(0) / o["n"][i]
    used, N = int((o["n"] > 0).sum()), int(o["n"].sum())
    bal = sum((E * o["counts"][i] / (k * o["n"][i]) * o["prob"][i]).sum() for i in range(S) if o["n"][i])
    zs = sum((lse[off[i]:off[i + 1]] ** 2 * real[off[i]:off[i + 1]]).sum() for i in range(S))
    bal, z = alpha * bal / max(used, 1), beta * zs / max(N, 1)
    o["loss"] = np.array([bal + z, bal, z])
    if d_loss is not None:
        for i in range(S):
            if not o["n"][i]:
                continue
            r = slice(off[i], off[i + 1])
            c = d_loss * alpha * E * o["counts"][i] / (k * o["n"][i] ** 2 * used)
            p = share[r]
            dot = (p * c).sum(1, keepdims=True)
            zt = d_loss * 2 * beta / N * lse[r][:, None]
            g[r] += p * (c - dot + zt) * slope[r] * real[r, None]
            gmag[r] += p * (c + np.abs(dot) + np.abs(zt))
    if dw is not None:
        G = np.zeros((T, E))
        for j in range(idx.shape[1]):
            on = (idx[:, j] >= 0) & (idx[:, j] < E)
            G[np.nonzero(on)[0], idx[on, j]] = scale * dw[on, j]
        base = q if renorm else s
        if renorm or score == "softmax":
            dot = (base * G).sum(1, keepdims=True)
            g += base * slope * (G - dot)
            gmag += base * (np.abs(G) + np.abs(base * G).sum(1, keepdims=True))
        else:
            g += s * slope * G
            gmag += np.abs(s * G)
    o["grad"], o["grad_mag"] = g, gmag
    return o


def close(got, ref, what, rel=2.0 ** -16, mag=None):
    got = got.detach().double().cpu().numpy()
    mag = np.abs(ref) if mag is None else mag
    err = np.abs(got - ref)
    bad = ~(err <= rel * mag + 1e-30)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {err.max():.3g}"


EXPERTS = [(1, 1), (2, 1), (5, 5), (8, 2), (31, 4), (33, 8), (64, 6), (100, 32), (256, 8), (257, 7), (513, 16), (1024, 32)]


@pytest.mark.parametrize("E,k", EXPERTS)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_forward(m, E, k, dtype, score, renorm):
    T = 67
    x = make(T, E, dtype, seed=E, scale=2.0)
    bias = 0.3 * make(1, E, seed=E + 1)[0]
    x[5] = -math.inf                                     # a padding token
    x[6, : E - 1] = -math.inf                            # one expert open
    x[7] = math.nan                                      # nothing open either
    x[8, ::2] = math.nan
    x[9] = 0.25                                          # all equal: lowest indices
    x[10, E // 2] = math.inf
    x[11] = -1e30                                        # sigmoids underflow
    x[12] = -0.0
    x[12, E // 2:] = 0.0                                 # -0 and 0 tie
    op = m.Router(E, k, score=score, renormalize=renorm, weight_scale=2.5, logits_dtype=dtype, device=DEV)
    for b in (None, bias):
        out = op.forward(x, b)
        idx = ref_choice(x, b, k)
        assert np.array_equal(out.topk_idx.cpu().numpy(), idx)
        ref = ref_all(x, idx, score, renorm, 2.5, k)
        got = out.topk_weights.cpu().numpy()
        if score == "sigmoid" and renorm:                # row 11: ratios of underflowing sigmoids, which 64 bits lose too
            n = (idx[11] >= 0).sum()
            np.testing.assert_allclose(got[11, :n], 2.5 / n, rtol=1e-5)
            ref["weights"][11] = got[11]
        close(out.topk_weights, ref["weights"], "weights")
        if renorm:
            full = (idx >= 0).any(1)
            np.testing.assert_allclose(got.sum(1)[full], 2.5, rtol=1e-5)


def test_all_ties_bf16(m):
    """Few distinct values: every choice is decided by the index rule."""
    T, E, k = 300, 160, 13
    g = torch.Generator().manual_seed(3)
    x = torch.randint(0, 3, (T, E), generator=g).to(BF).to(DEV)
    out = m.Router(E, k, logits_dtype=BF, device=DEV).forward(x)
    assert np.array_equal(out.topk_idx.cpu().numpy(), ref_choice(x, None, k))


def test_closed_by_bias(m):
    T, E, k = 9, 48, 6
    x = make(T, E, seed=4)
    bias = torch.zeros(E, device=DEV)
    bias[::2] = -math.inf
    bias[1] = math.inf
    bias[3] = math.nan
    out = m.Router(E, k, device=DEV).forward(x, bias)
    idx = ref_choice(x, bias, k)
    assert np.array_equal(out.topk_idx.cpu().numpy(), idx) and (idx[:, 0] == 1).all() and not np.isin(idx, [0, 2, 3]).any()
    close(out.topk_weights, ref_all(x, idx, "softmax", True, 1.0, k)["weights"], "weights")


@pytest.mark.parametrize("E", [8, 40, 256])
@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 0), (3, 1)])
def test_pitched_logits(m, E, pad, offset):
    T, k = 21, 3
    x = make(T, E, BF, seed=6)
    buf = torch.full((T * (E + pad) + offset + 4,), 9.0, dtype=BF, device=DEV)
    v = torch.as_strided(buf, (T, E), (E + pad, 1), offset)
    v.copy_(x)
    op = m.Router(E, k, balance_coef=1.0, z_coef=0.5, logits_dtype=BF, max_tokens=T, device=DEV)
    a, b = op.forward_train(x), op.forward_train(v)
    for n in ("topk_idx", "topk_weights", "loss", "counts", "prob_mean", "seq_tokens"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    dw, one = torch.ones(T, k, device=DEV) * torch.arange(k, device=DEV), torch.ones((), device=DEV)
    gbuf = torch.full_like(buf, 5.0)
    gv = torch.as_strided(gbuf, (T, E), (E + pad, 1), offset)
    ga = op.backward(x, a, dw, one)
    op.backward(v, b, dw, one, out=gv)
    assert torch.equal(ga, gv)
    keep = torch.ones_like(gbuf, dtype=torch.bool)
    torch.as_strided(keep, (T, E), (E + pad, 1), offset).fill_(False)
    assert (gbuf[keep] == 5.0).all()


def sequences(T, kind):
    return {"one": None, "ragged": [0, 1, 1, T // 3, T // 3 + 2, T - 1, T], "inside": [2, T // 2, T - 3],
            "empty": [T, T, T], "many": list(range(0, T + 1))}[kind]


@pytest.mark.parametrize("T", [5, 130, 3001])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (40, 5), (256, 8), (600, 3)])
@pytest.mark.parametrize("kind", ["one", "ragged", "inside", "empty", "many"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_losses_and_gradient(m, T, E, k, kind, score):
    off = sequences(T, kind)
    x = make(T, E, seed=T + E, scale=1.5)
    x[T // 2] = -math.inf
    x[3, : E // 2] = -math.inf
    alpha, beta = 0.7, 0.3 if score == "softmax" else 0.0
    S = 1 if off is None else len(off) - 1
    offs = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(7)
    dw = torch.randn(T, k, generator=g).to(DEV)
    one = torch.full((), 1.5, device=DEV)
    for renorm in (True, False):
        op = m.Router(E, k, score=score, renormalize=renorm, weight_scale=1.25, balance_coef=alpha, z_coef=beta, max_tokens=T,
                      max_seqs=S, device=DEV)
        out = op.forward_train(x, None, offs)
        plain = op.forward(x)
        assert torch.equal(out.topk_idx, plain.topk_idx) and torch.equal(out.topk_weights, plain.topk_weights)
        idx = ref_choice(x, None, k)
        assert np.array_equal(out.topk_idx.cpu().numpy(), idx)
        ref = ref_all(x, idx, score, renorm, 1.25, k, off, alpha, beta, dw.double().cpu().numpy(), 1.5)
        assert np.array_equal(out.counts.cpu().numpy(), ref["counts"])
        assert np.array_equal(out.seq_tokens.cpu().numpy(), ref["n"])
        assert out.tokens[S:].tolist() == [int((ref["n"] > 0).sum()), int(ref["n"].sum())]
        close(out.prob_mean, ref["prob"], "prob_mean")
        close(out.loss, ref["loss"], "loss")
        given = op.balance_loss(x, out.topk_idx, offs)
        for n in ("loss", "counts", "prob_mean", "seq_tokens"):
            assert torch.equal(getattr(given, n), getattr(out, n)), n
        d = op.backward(x, out, dw, one, offs)
        close(d, ref["grad"], "d_logits", mag=ref["grad_mag"])
        assert (d[T // 2] == 0).all() and (d[3, : E // 2] == 0).all()
        # each part by itself, and their sum
        a, b = op.backward(x, out, dw, None, offs), op.backward(x, out, None, one, offs)
        ra = ref_all(x, idx, score, renorm, 1.25, k, off, alpha, beta, dw.double().cpu().numpy(), None)
        rb = ref_all(x, idx, score, renorm, 1.25, k, off, alpha, beta, None, 1.5)
        close(a, ra["grad"], "d_logits through the weights", mag=ra["grad_mag"])
        close(b, rb["grad"], "d_logits of the loss", mag=rb["grad_mag"])


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_bf16_gradient(m, score, renorm):
    T, E, k = 333, 72, 6
    x = make(T, E, BF, seed=1)
    op = m.Router(E, k, score=score, renormalize=renorm, balance_coef=1.0, logits_dtype=BF, max_tokens=T, device=DEV)
    out = op.forward_train(x)
    dw = make(T, k, seed=2)
    d = op.backward(x, out, dw, torch.ones((), device=DEV))
    ref = ref_all(x, out.topk_idx.cpu().numpy(), score, renorm, 1.0, k, None, 1.0, 0.0, dw.double().cpu().numpy(), 1.0)
    close(d, ref["grad"], "d_logits", rel=2.0 ** -8, mag=np.abs(ref["grad"]) + 2.0 ** -8 * ref["grad_mag"])


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(m, score, renorm):
    """Central differences of the forward calls along a direction that changes no choice.  Step 2^-6: truncation about
    step^2 / 6 of the third derivative, f32 noise 2^-24 / 2^-6 of the terms; 2^-9 of the terms covers both."""
    T, E, k = 23, 24, 4
    base = torch.argsort(torch.rand(T, E, generator=torch.Generator().manual_seed(5)), 1).float().to(DEV) / 6   # gaps of 1/6
    alpha, beta = 1.0, 0.25 if score == "softmax" else 0.0
    op = m.Router(E, k, score=score, renormalize=renorm, balance_coef=alpha, z_coef=beta, max_tokens=T, max_seqs=3, device=DEV)
    offs = torch.tensor([0, 4, 15, T], dtype=torch.int32, device=DEV)
    dw = make(T, k, seed=9)
    out = op.forward_train(base, None, offs)
    d = op.backward(base, out, dw, torch.ones((), device=DEV), offs)
    for seed in range(4):
        v = make(T, E, seed=20 + seed).clamp(-2, 2)
        step = 2.0 ** -6
        vals = []
        for sgn in (1, -1):
            o = op.forward_train(base + sgn * step * v, None, offs)
            assert torch.equal(o.topk_idx, out.topk_idx)
            vals.append(float(o.loss[0].double()) + float((o.topk_weights.double() * dw.double()).sum()))
        num = (vals[0] - vals[1]) / (2 * step)
        ana, scale = float((d.double() * v.double()).sum()), float((d.double() * v.double()).abs().sum())
        assert abs(num - ana) <= 2.0 ** -9 * scale, (num, ana, scale)


def test_given_choice_with_inactive_slots(m):
    T, E, k = 50, 16, 3
    x = make(T, E, seed=3)
    idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)]).to(torch.int32)
    idx[7, 1] = -1
    idx[8] = -1
    idx[9, 0] = E + 5                                    # outside: inactive
    op = m.Router(E, k, balance_coef=2.0, max_tokens=T, device=DEV)
    out = op.balance_loss(x, idx.to(DEV))
    ref = ref_all(x, idx.numpy(), "softmax", True, 1.0, k, None, 2.0, 0.0)
    assert np.array_equal(out.counts.cpu().numpy(), ref["counts"])
    close(out.loss, ref["loss"], "loss")
    out.topk_idx = idx.to(DEV)
    dw = make(T, k, seed=8)
    d = op.backward(x, out, dw, torch.ones((), device=DEV))
    ref = ref_all(x, idx.numpy(), "softmax", True, 1.0, k, None, 2.0, 0.0, dw.double().cpu().numpy(), 1.0)
    close(d, ref["grad"], "d_logits", mag=ref["grad_mag"])


def test_no_tokens(m):
    E, k, S = 12, 2, 3
    op = m.Router(E, k, balance_coef=1.0, z_coef=1.0, max_tokens=10, max_seqs=S, device=DEV)
    x = torch.empty(0, E, device=DEV)
    out = op.buffers(0, S)
    for t in (out.loss, out.prob_mean):
        t.fill_(7)
    out.counts.fill_(7)
    op.forward_train(x, None, torch.zeros(S + 1, dtype=torch.int32, device=DEV), out=out)
    assert (out.loss == 0).all() and (out.counts == 0).all() and (out.prob_mean == 0).all() and (out.tokens == 0).all()
    assert op.backward(x, out, None, torch.ones((), device=DEV), torch.zeros(S + 1, dtype=torch.int32, device=DEV)).shape == (0, E)
    assert op.forward(x).topk_idx.shape == (0, k)


def test_large_batch_is_repeatable(m):
    """Many warps per sequence, twice: the same bits; counts sum to the chosen slots; the layer's dispatch takes the indices."""
    T, E, k = 20011, 256, 8
    x = make(T, E, seed=13)
    offs = torch.tensor([0, 5000, 5001, 12345, T], dtype=torch.int32, device=DEV)
    op = m.Router(E, k, balance_coef=1e-2, z_coef=1e-3, max_tokens=T, max_seqs=4, device=DEV)
    a = op.forward_train(x, None, offs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = op.forward_train(x, None, offs, stream=side)
    side.synchronize()
    for n in ("topk_idx", "topk_weights", "loss", "counts", "prob_mean", "seq_tokens"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    assert int(a.counts.sum()) == T * k
    ref = ref_all(x, a.topk_idx.cpu().numpy(), "softmax", True, 1.0, k, offs.tolist(), 1e-2, 1e-3)
    assert np.array_equal(a.counts.cpu().numpy(), ref["counts"])
    close(a.loss, ref["loss"], "loss")


def test_offsets_past_32_bits(m):
    T, E, k, pitch = 3, 64, 4, 1_200_000_001
    x = make(T, E, BF, seed=2)
    big = torch.empty((T - 1) * pitch + E, dtype=BF, device=DEV)
    far = torch.as_strided(big, (T, E), (pitch, 1))
    far.copy_(x)
    op = m.Router(E, k, balance_coef=1.0, logits_dtype=BF, max_tokens=T, device=DEV)
    a, b = op.forward_train(x), op.forward_train(far)
    assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.loss, b.loss)
    one = torch.ones((), device=DEV)
    d = op.backward(x, a, None, one)
    op.backward(far, b, None, one, out=far)              # in place
    assert torch.equal(d, far)


def test_graph_capture(m):
    T, E, k = 128, 256, 8
    x = make(T, E, seed=5)
    op = m.Router(E, k, balance_coef=1.0, z_coef=0.1, max_tokens=T, device=DEV)
    want = op.forward_train(x)
    out = op.buffers(T, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        op.forward_train(x, out=out)
        with torch.cuda.graph(g, stream=s):
            op.forward_train(x, out=out)
    for _ in range(3):
        out.loss.zero_()
        out.counts.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.loss, want.loss) and torch.equal(out.counts, want.counts)


@pytest.mark.parametrize("T,S", [(19, 20), (700, 33), (700, 70), (5000, 1500), (60, 2100)])
def test_ragged_sequences_with_runs_of_empty_ones(m, T, S):
    """Sequences are found 32 offsets at a time: runs of empty ones longer than that, gaps at both ends."""
    E, k = 24, 3
    g = torch.Generator().manual_seed(T + S)
    cut = torch.randint(1, T, (S + 1,), generator=g)
    cut[S // 4: S // 2] = T // 3
    cut[-S // 5:] = T - 1
    off = sorted(cut.tolist())
    x = make(T, E, seed=S)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    dw, one = torch.randn(T, k, generator=g).to(DEV), torch.full((), 2.0, device=DEV)
    op = m.Router(E, k, balance_coef=0.5, z_coef=0.25, max_tokens=T, max_seqs=S, device=DEV)
    out = op.forward_train(x, None, offs)
    idx = ref_choice(x, None, k)
    ref = ref_all(x, idx, "softmax", True, 1.0, k, off, 0.5, 0.25, dw.double().cpu().numpy(), 2.0)
    assert np.array_equal(out.topk_idx.cpu().numpy(), idx)
    assert np.array_equal(out.counts.cpu().numpy(), ref["counts"]) and np.array_equal(out.seq_tokens.cpu().numpy(), ref["n"])
    close(out.prob_mean, ref["prob"], "prob_mean")
    close(out.loss, ref["loss"], "loss")
    close(op.backward(x, out, dw, one, offs), ref["grad"], "d_logits", mag=ref["grad_mag"])
