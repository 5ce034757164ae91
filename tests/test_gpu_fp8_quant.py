"""Fp8Quant against the definition in 64 bits: rows, columns, both and blocks, ends inside a group, zero, tiny, infinite and NaN
groups, pitches; SwiGLU and its gradient (the formula in 64 bits is checked against differences); repeats, streams, capture.

Tolerances: scales are one rounded quotient (2^-23), codes the nearest E4M3 of a quotient within 2^-22 (fp8_ref.close_codes).
SwiGLU's f32 error: the sigmoid within 2^-20 (exponential within 2 units, its argument exact, a quotient within 2) or, where it is
below the normal numbers, 2^-149, the smallest one; products 2^-24 each, or 2^-149; the gradient's factor s (1 + g (1 - s)) is a sum of terms whose magnitudes s and |g| s (1 - s) bound it."""
import math

import pytest
import torch

from fp8_ref import BF, DEV, F32, close_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def tokens(T, H, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(T, H, generator=g) * torch.exp2(3 * torch.randn(T, 1, generator=g)) * torch.exp2(3 * torch.randn(1, H, generator=g))
    return v.to(dt).to(DEV)


def check(o, v, err, what=""):
    if o.codes is not None:
        close_codes(o.codes, o.sf, v, err, 1, 128, what + " rows")
    if o.col_codes is not None:
        close_codes(o.col_codes, o.col_sf, v, err, 128, 1, what + " columns")


FORMS = [dict(rows=True, cols=False), dict(rows=False, cols=True), dict(rows=True, cols=True)]
TS = [1, 2, 31, 32, 33, 127, 128, 129, 300]


@pytest.mark.parametrize("H", [16, 112, 128, 144, 400, 1024, 4112])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_tokens(m, H, dt):
    op = m.Fp8Quant(H, dtype=dt, device=DEV)
    for T in TS:
        v = tokens(T, H, dt, T)
        zero = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for f in FORMS:
            o = op.forward(v, **f)
            assert (o.codes is not None) == f["rows"] and (o.col_codes is not None) == f["cols"]
            check(o, v.double(), zero, f"T={T}")


@pytest.mark.parametrize("N,H", [(1, 16), (16, 144), (128, 128), (129, 272), (300, 1040), (1000, 4112)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_weights(m, N, H, dt):
    w = tokens(N, H, dt, 3)
    o = m.Fp8Quant(H, dtype=dt, device=DEV).weights(w)
    close_codes(o.codes, o.sf, w.double(), torch.zeros(N, H, dtype=torch.float64, device=DEV), 128, 128)


def ref_swiglu(v, clamp):
    H = v.shape[1] // 2
    g, u = v[:, :H].double().clamp(-clamp, clamp), v[:, H:].double().clamp(-clamp, clamp)
    y = g * torch.sigmoid(g) * u
    return y, 2.0 ** -19 * y.abs() + 2.0 ** -148 * (g * u).abs() + 2.0 ** -148


def ref_grad(d, v, clamp):
    H = v.shape[1] // 2
    g0, u0, d = v[:, :H].double(), v[:, H:].double(), d.double()
    g, u = g0.clamp(-clamp, clamp), u0.clamp(-clamp, clamp)
    s = torch.sigmoid(g)
    dg = torch.where(g0.abs() > clamp, torch.zeros_like(g), d * u * s * (1 + g * (1 - s)))
    du = torch.where(u0.abs() > clamp, torch.zeros_like(g), d * g * s)
    eg = (2.0 ** -19 * s + 2.0 ** -148) * (d * u).abs() * (1 + g.abs()) + 2.0 ** -148
    return torch.cat([dg, du], 1), torch.cat([eg, 2.0 ** -19 * du.abs() + 2.0 ** -148 * (d * g).abs() + 2.0 ** -148], 1)


@pytest.mark.parametrize("H", [128, 640, 2048])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("clamp", [math.inf, 1.5], ids=["open", "clamped"])
def test_swiglu_and_its_gradient(m, H, dt, clamp):
    op = m.Fp8Quant(H, act="swiglu", dtype=dt, act_clamp=clamp, device=DEV)
    for T in TS:
        v, d = tokens(T, 2 * H, dt, T), tokens(T, H, dt, T + 1)
        for f in FORMS:
            check(op.forward(v, **f), *ref_swiglu(v, clamp), f"T={T}")
            check(op.backward(d, v, **f), *ref_grad(d, v, clamp), f"T={T} grad")


def test_the_gradients_formula_is_the_difference():
    g = torch.Generator().manual_seed(0)
    v, d = 3 * torch.randn(7, 64, generator=g).double(), torch.randn(7, 32, generator=g).double()
    grad, _ = ref_grad(d, v, 2.0)
    h = 1e-6
    for j in range(64):
        e = torch.zeros_like(v)
        e[:, j] = h
        diff = (d * (ref_swiglu(v + e, 2.0)[0] - ref_swiglu(v - e, 2.0)[0])).sum(1) / (2 * h)
        assert (diff - grad[:, j]).abs().max() <= 1e-7


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_zero_tiny_infinite_and_nan_groups(m, dt):
    T, H = 260, 400
    v = tokens(T, H, dt, 5)
    v[1] = 0
    v[:, 130] = 0
    v[3] = torch.ldexp(torch.randn(H, generator=torch.Generator().manual_seed(1)), torch.tensor(-125)).to(dt).to(DEV)   # below 2^-100
    v[:, 140] = torch.ldexp(torch.randn(T, generator=torch.Generator().manual_seed(2)), torch.tensor(-112)).to(dt).to(DEV)
    v[5, 7] = math.nan
    v[200, 9] = -math.inf
    o = m.Fp8Quant(H, dtype=dt, device=DEV).forward(v, rows=True, cols=True)
    # row 1 is zero but for column 140, column 130 but for row 3
    none = v == 0
    assert (o.sf[1, [0, 2, 3]] == 0).all() and o.sf[1, 1] > 0 and ((o.codes & 127) == 0)[none].all()
    assert (o.col_sf[1:, 130] == 0).all() and o.col_sf[0, 130] > 0 and ((o.col_codes & 127) == 0)[none].all()
    clean = v.double()
    # a NaN is a NaN's code and takes no part in its group's scale
    assert (o.codes[5, 7] & 127) == 127 and (o.col_codes[5, 7] & 127) == 127
    clean[5, 7] = 0
    # an infinity: the scale infinity, every value of its group a NaN
    assert math.isinf(o.sf[200, 0]) and math.isinf(o.col_sf[1, 9])
    value = o.codes.view(torch.float8_e4m3fn).double() * o.sf.double().repeat_interleave(128, 1)[:, :H]
    assert torch.isnan(value[200, :128]).all() and torch.isfinite(value[200, 128:]).all()
    value = o.col_codes.view(torch.float8_e4m3fn).double() * o.col_sf.double().repeat_interleave(128, 0)[:T]
    assert torch.isnan(value[128:256, 9]).all() and torch.isfinite(value[:128, 9]).all()
    keep = torch.ones(T, H, dtype=torch.bool, device=DEV)
    keep[5, 7] = False
    # subnormal scales keep 2^-149 of themselves absolutely: 448 times that of a value, and half a step
    for codes, sf, rows in ((o.codes, o.sf.double().repeat_interleave(128, 1)[:, :H], True),
                            (o.col_codes, o.col_sf.double().repeat_interleave(128, 0)[:T], False)):
        on = keep.clone()
        if rows:
            on[200, :128] = False
        else:
            on[128:256, 9] = False
        off = (codes.view(torch.float8_e4m3fn).double() * sf - clean).abs()
        tol = (2.0 ** -4 * clean.abs()).maximum(2.0 ** -10 * sf) * 1.001 + 448 * 2.0 ** -148
        assert (off[on] <= tol[on]).all()


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_pitches(m, dt):
    T, H = 200, 272
    es = 16 // (2 if dt is BF else 4)
    v = tokens(T, H, dt, 8)
    op = m.Fp8Quant(H, dtype=dt, device=DEV)
    ref = op.forward(v, cols=True)
    buf = torch.full((T, H + 3 * es), math.nan, dtype=dt, device=DEV)
    view = buf[:, es:es + H]
    view.copy_(v)
    o = op.forward(view, cols=True)
    for n in ("codes", "sf", "col_codes", "col_sf"):
        assert torch.equal(getattr(o, n), getattr(ref, n))
    with pytest.raises(m.MoEError):
        op.forward(buf[:, 1:1 + H])       # rows that are not 16-byte aligned


def test_no_rows(m):
    o = m.Fp8Quant(128, device=DEV).forward(torch.empty(0, 128, dtype=BF, device=DEV), cols=True)
    assert o.codes.shape == (0, 128) and o.col_sf.shape == (0, 128)
    assert m.Fp8Quant(128, device=DEV).weights(torch.empty(0, 128, dtype=BF, device=DEV)).codes.shape == (0, 128)


def test_past_2_31_elements(m):
    T, H = 16400, 131088
    v = torch.zeros(T, H, dtype=BF, device=DEV)
    rows = [0, 16381, 16382, 16383, T - 1]
    v[rows] = tokens(len(rows), H, BF, 1)
    o = m.Fp8Quant(H, device=DEV).forward(v, cols=True)
    zero = torch.zeros(len(rows), H, dtype=torch.float64, device=DEV)
    close_codes(o.codes[rows], o.sf[rows], v[rows].double(), zero, 1, 128)
    last = o.col_codes[16384:], o.col_sf[128:]
    close_codes(*last, v[16384:].double(), torch.zeros(16, H, dtype=torch.float64, device=DEV), 128, 1)


@pytest.mark.parametrize("T", [1, 300])
def test_repeats_streams_and_capture(m, T):
    H = 640
    op, v, d = m.Fp8Quant(H, act="swiglu", device=DEV), tokens(T, 2 * H, BF, 1), tokens(T, H, BF, 2)
    flat = lambda o: [getattr(o, n) for n in ("codes", "sf", "col_codes", "col_sf")]  # noqa: E731
    run = lambda a, b, s=None: (op.forward(v, cols=True, out=a, stream=s), op.backward(d, v, out=b, stream=s))  # noqa: E731
    first = [t.clone() for o in run(None, None) for t in flat(o)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = [t for o in run(None, None, s) for t in flat(o)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, side))
    out = op.buffers(T, cols=True), op.buffers(T, cols=True, grad=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        run(*out)
        with torch.cuda.graph(g, stream=s):
            run(*out)
    for o in out:
        for t in flat(o):
            t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, [t for o in out for t in flat(o)]))
