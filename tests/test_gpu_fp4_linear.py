"""Fp4Linear against products in 64 bits: every token count, odd widths, short
and long K, extreme scales and inputs, both activations, added inputs, pitches.

Tolerances.  Weights are exact (two significant bits times a power of two) and
so are bf16 inputs, products in f32 are exact; sums of K of them in f32, in
blocks of at most 32 joined by a chain, stay within 2^-18 of the sum of their
magnitudes.  The output is one rounding more: 2^-8 of the value in bf16.
SwiGLU multiplies: its relative error is that of its factors, the sigmoid's
slope is below 1, so the bound is taken through the product.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def make(N, K, seed=0, lo=118, hi=124):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    sf = torch.randint(lo, hi, (N, K // 32), generator=g).to(torch.uint8)
    return w, sf


def dense(w, sf):
    w = w.numpy()
    v = np.empty((w.shape[0], 2 * w.shape[1]))
    v[:, 0::2], v[:, 1::2] = GRID[w & 15], GRID[w >> 4]
    return v * np.repeat(np.ldexp(1.0, sf.numpy().astype(np.int32) - 127), 32, axis=1)


def ref(x, W, act=None, clamp=math.inf, add=None):
    """(value, bound on the f32 value's error)"""
    x = x.double().cpu().numpy()
    y, mag = x @ W.T, np.abs(x) @ np.abs(W).T
    err = 2.0 ** -18 * mag
    if act == "swiglu":
        n = y.shape[1] // 2
        g, u, eg, eu = np.clip(y[:, :n], -clamp, clamp), np.clip(y[:, n:], -clamp, clamp), err[:, :n], err[:, n:]
        s = 1 / (1 + np.exp(-g))
        y = g * s * u
        err = (1.1 * eg * np.abs(u) + np.abs(g * s) * eu + eg * eu) + 2.0 ** -20 * np.abs(y)
    if add is not None:
        a = add.double().cpu().numpy()
        err = err + 2.0 ** -22 * (np.abs(y) + np.abs(a))
        y = y + a
    return y, err


def close(got, y, err, what=""):
    u = 2.0 ** -8 if got.dtype == BF else 2.0 ** -23
    g = got.double().cpu().numpy()
    assert g.shape == y.shape
    tol = u * np.abs(y) + err * (1 + u) + 1e-38
    bad = ~(np.abs(g - y) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {(np.abs(g - y) / tol).max():.3g} x tolerance"


def build(m, N, K, w, sf, **kw):
    op = m.Fp4Linear(K, N, device=DEV, **kw)
    op.transform_weights(w.to(DEV), sf.to(DEV))
    return op


@pytest.mark.parametrize("N,K", [(1, 32), (3, 64), (16, 96), (17, 128), (31, 160), (100, 1024), (129, 2080), (77, 7168), (1000, 480),
                                 (33, 14336)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_every_token_count(m, N, K, act):
    N = 2 * N if act else N
    w, sf = make(N, K, seed=N + K)
    W = dense(w, sf)
    ops = {dt: build(m, N, K, w, sf, act=act, out_dtype=dt) for dt in (BF, F32)}
    g = torch.Generator().manual_seed(1)
    for M in list(range(1, 17)):
        x = torch.randn(M, K, generator=g).to(BF).to(DEV)
        for dt, op in ops.items():
            y, err = ref(x, W, act)
            close(op.forward(x), y, err, f"M={M} {dt}")


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_add_pitches_and_in_place(m, M, dt):
    N, K = 203, 288
    w, sf = make(N, K, seed=5)
    op = build(m, N, K, w, sf, out_dtype=dt)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(M, K, generator=g).to(BF).to(DEV)
    add = torch.randn(M, N, generator=g).to(dt).to(DEV)
    y, err = ref(x, dense(w, sf), add=add)
    close(op.forward(x, add=add), y, err)
    out = add.clone()
    op.forward(x, add=out, out=out)
    close(out, y, err, "in place")
    for pad, offset in ((1, 1), (3, 0), (8, 0), (8, 8)):
        xb = torch.full((M * (K + pad) + offset,), 3.0, dtype=BF, device=DEV)
        xv = torch.as_strided(xb, (M, K), (K + pad, 1), offset)
        xv.copy_(x)
        yb = torch.full((M * (N + pad) + offset,), 5.0, dtype=dt, device=DEV)
        yv = torch.as_strided(yb, (M, N), (N + pad, 1), offset)
        op.forward(xv, add=add, out=yv)
        close(yv, y, err, f"pitch +{pad}")
        keep = torch.ones_like(yb, dtype=torch.bool)
        torch.as_strided(keep, (M, N), (N + pad, 1), offset).fill_(False)
        assert (yb[keep] == 5.0).all()


@pytest.mark.parametrize("M", [1, 5, 12])
def test_extreme_scales_and_inputs(m, M):
    """Scale codes from 0 (2^-127) to 254 (2^127), inputs from 2^-60 to 2^60, rows and columns of zeros."""
    N, K = 96, 1024
    w, _ = make(N, K, seed=11)
    rng = np.random.default_rng(3)
    sf = torch.from_numpy(np.repeat(rng.integers(0, 255, (N, 1)), K // 32, axis=1).astype(np.uint8))
    sf += torch.from_numpy(rng.integers(0, 2, (N, K // 32)).astype(np.uint8)) * (sf < 254)
    sf[0], sf[1], sf[2] = 0, 254, 1
    w[3] = 0
    w[4] = 0x88                                           # negative zeros
    g = torch.Generator().manual_seed(4)
    x = torch.randn(M, K, generator=g)
    if M > 1:
        x[0] = 0
        x[1] *= 2.0 ** 60
        x[2] *= 2.0 ** -60
        x[3] = torch.ldexp(x[3], torch.randint(-40, 40, (K,), generator=g))
    x = x.to(BF).to(DEV)
    W = dense(w, sf)
    y, err = ref(x, W)
    got = build(m, N, K, w, sf, out_dtype=F32).forward(x).double().cpu().numpy()
    big = 2.0 ** 18 * err > 1e38                          # partial sums may pass the f32 range
    # subnormal f32 partial sums keep 2^-149 absolutely; a scale of 2^-127 multiplies them after the sum
    tol = 2.0 ** -23 * np.abs(y) + err * (1 + 2.0 ** -20) + 2.0 ** -126
    assert (np.abs(got - y)[~big] <= tol[~big]).all(), (np.abs(got - y) / tol)[~big].max()
    assert (got[:, 3] == 0).all() and (got[:, 4] == 0).all()


def test_swiglu_clamp(m):
    N, K, M = 64, 256, 6
    w, sf = make(N, K, seed=9, lo=124, hi=128)
    op = build(m, N, K, w, sf, act="swiglu", out_dtype=F32, act_clamp=4.0)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(6)).to(BF).to(DEV)
    y, err = ref(x, dense(w, sf), "swiglu", 4.0)
    close(op.forward(x), y, err)
    assert np.abs(y).max() <= 16.0


def test_non_finite_inputs_stay_in_their_rows(m):
    N, K, M = 50, 512, 9
    w, sf = make(N, K, seed=10)
    w |= 0x11                                             # no zero weights
    op = build(m, N, K, w, sf, out_dtype=F32)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(6)).to(BF).to(DEV)
    clean = op.forward(x)
    x[2, 100] = math.nan
    x[5, 3] = math.inf
    out = op.forward(x)
    keep = [0, 1, 3, 4, 6, 7, 8]
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[2]).all() and not torch.isfinite(out[5]).any()


def test_no_tokens_too_many_and_no_weights(m):
    op = m.Fp4Linear(64, 8, device=DEV)
    with pytest.raises(m.MoEError) as e:
        op.forward(torch.zeros(1, 64, dtype=BF, device=DEV))
    assert e.value.code == m.MOE_ERR_NOT_READY
    w, sf = make(8, 64)
    op.transform_weights(w.to(DEV), sf.to(DEV))
    assert op.forward(torch.zeros(0, 64, dtype=BF, device=DEV)).shape == (0, 8)
    with pytest.raises(m.MoEError) as e:
        op.forward(torch.zeros(17, 64, dtype=BF, device=DEV))
    assert e.value.code == m.MOE_ERR_UNSUPPORTED


def test_repeatable_streams_and_graph(m):
    N, K, M = 2048, 7168, 3
    w, sf = make(N, K, seed=20)
    op = build(m, N, K, w, sf)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(6)).to(BF).to(DEV)
    a = op.forward(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = op.forward(x, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    out = op.buffers(M)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        op.forward(x, out=out)
        with torch.cuda.graph(g, stream=s):
            op.forward(x, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)
