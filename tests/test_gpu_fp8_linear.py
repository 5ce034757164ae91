"""Fp8Linear against products in 64 bits: token counts and sizes on both sides of every tile and variant, blocks that end early,
SwiGLU and quantised outputs, added inputs, pitches, zero and infinite scales, NaN codes, matrices past 2^31 elements; gradients
against the formulas and against differences; repeats, streams, capture.  Tolerances: fp8_ref.py."""
import math

import pytest
import torch

from fp8_ref import BF, DEV, F32, close, close_codes, product, random_codes, swiglu, up, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    yield mod
    assert mod.lib().moe_fp8_linear_status() == mod.MOE_OK


SIZES = [(16, 16), (128, 128), (144, 272), (272, 144), (1040, 656), (400, 2064)]
TOKENS = [1, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 300]
# enough 256 x 256 tiles for CTA pairs, ends inside tiles and blocks
WIDE = [(2500, 1040, 400), (300, 9744, 272), (2561, 1296, 144), (1000, 5136, 16), (129, 10240, 1040)]


def forward_inputs(T, N, K, seed=0):
    return (*random_codes(T, K, 1, 128, seed), *random_codes(N, K, 128, 128, seed + 1, scale=1 / K))


def ref_forward(x, x_sf, w, w_sf):
    return product(values(x, x_sf, 1, 128), values(w, w_sf, 128, 128), up(x.shape[1]))


@pytest.mark.parametrize("N,K", SIZES)
def test_forward(m, N, K):
    ops = [m.Fp8Linear(K, N, out_dtype=dt, device=DEV) for dt in (BF, F32)]
    for T in TOKENS:
        a = forward_inputs(T, N, K, T)
        y, err = ref_forward(*a)
        for op in ops:
            close(op.forward(*a), y, err, f"T={T} {op.out_dtype}")


@pytest.mark.parametrize("T,N,K", WIDE)
def test_forward_wide(m, T, N, K):
    a = forward_inputs(T, N, K)
    y, err = ref_forward(*a)
    for dt in (BF, F32):
        close(m.Fp8Linear(K, N, out_dtype=dt, device=DEV).forward(*a), y, err, str(dt))


@pytest.mark.parametrize("T,N,K", [(1, 256, 128), (3, 512, 400), (16, 256, 1040), (17, 768, 272), (64, 512, 144), (65, 256, 528),
                                   (200, 1024, 656), (129, 5120, 272), (2561, 1024, 144), (1000, 4096, 400)])
@pytest.mark.parametrize("clamp", [math.inf, 0.75], ids=["open", "clamped"])
def test_swiglu_and_its_codes(m, T, N, K, clamp):
    a = forward_inputs(T, N, K, 7)
    y, err = swiglu(*ref_forward(*a), clamp)
    for dt in (BF, F32):
        close(m.Fp8Linear(K, N, act="swiglu", out_dtype=dt, act_clamp=clamp, device=DEV).forward(*a), y, err, str(dt))
    o = m.Fp8Linear(K, N, act="swiglu", quant="fp8", act_clamp=clamp, device=DEV).forward(*a)
    close_codes(o.codes, o.sf, y, err, 1, 128)


@pytest.mark.parametrize("T,N,K", [(t, n, k) for t in (1, 16, 17, 33, 64, 65, 129, 300) for n, k in ((16, 16), (144, 272), (656, 400), (128, 1040))]
                         + [(2500, 400, 1040), (300, 272, 9744), (2561, 144, 1296), (1000, 16, 5136)])
def test_input_gradient(m, T, N, K):
    dy, dy_sf = random_codes(T, N, 1, 128, T)
    w, w_sf = random_codes(N, K, 128, 128, 5, scale=1 / N)
    dx, err = product(values(dy, dy_sf, 1, 128), values(w, w_sf, 128, 128).t(), up(N))
    for dt in (BF, F32):
        close(m.Fp8Linear(K, N, out_dtype=dt, device=DEV).backward_input(dy, dy_sf, w, w_sf), dx, err, str(dt))


@pytest.mark.parametrize("T,N,K", [(t, n, k) for t in (1, 127, 128, 129, 257, 1000) for n, k in ((16, 16), (144, 272), (272, 144), (400, 1040))]
                         + [(300, 2560, 1040), (1, 2576, 1040), (129, 1296, 2560), (1025, 1040, 2576)])
def test_weight_gradient(m, T, N, K):
    dy, dy_sf = random_codes(T, N, 128, 1, T)
    x, x_sf = random_codes(T, K, 128, 1, 5)
    dw, err = product(values(dy, dy_sf, 128, 1).t(), values(x, x_sf, 128, 1).t(), up(T))
    op = m.Fp8Linear(K, N, device=DEV)
    close(op.backward_weight(dy, dy_sf, x, x_sf), dw, err)
    add = torch.randn(N, K, generator=torch.Generator().manual_seed(1)).to(DEV)
    both, err = dw + add.double(), err + 2.0 ** -23 * (dw.abs() + add.abs().double())
    close(op.backward_weight(dy, dy_sf, x, x_sf, add=add), both, err)
    op.backward_weight(dy, dy_sf, x, x_sf, add=add, out=add)
    close(add, both, err, "in place")


@pytest.mark.parametrize("T,N,K", [(3, 144, 272), (33, 144, 272), (100, 272, 144), (2500, 1040, 144)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_add_pitches_and_in_place(m, T, N, K, dt):
    x, x_sf, w, w_sf = forward_inputs(T, N, K, 3)
    op = m.Fp8Linear(K, N, out_dtype=dt, device=DEV)
    add = torch.randn(T, N, generator=torch.Generator().manual_seed(2)).to(dt).to(DEV)
    y, err = ref_forward(x, x_sf, w, w_sf)
    y, err = y + add.double(), err + 2.0 ** -23 * (y.abs() + add.abs().double())
    close(op.forward(x, x_sf, w, w_sf, add=add), y, err)
    same = add.clone()
    op.forward(x, x_sf, w, w_sf, add=same, out=same)
    close(same, y, err, "in place")
    es = 16 // add.element_size()
    for pad, offset in ((es, 0), (2 * es, es), (3 * es, 2 * es)):     # 16-byte and 32-byte aligned rows
        xb = torch.full((T * (K + 16 * pad) + 16,), 0x7F, dtype=torch.uint8, device=DEV)     # NaN codes around the rows
        xv = torch.as_strided(xb, (T, K), (K + 16 * pad, 1), 16)
        xv.copy_(x)
        yb = torch.full((T * (N + pad) + offset,), 5.0, dtype=dt, device=DEV)
        yv = torch.as_strided(yb, (T, N), (N + pad, 1), offset)
        av = torch.as_strided(yb.clone(), (T, N), (N + pad, 1), offset)
        av.copy_(add)
        op.forward(xv, x_sf, w, w_sf, add=av, out=yv)
        close(yv, y, err, f"pitch +{pad}")
        keep = torch.ones_like(yb, dtype=torch.bool)
        torch.as_strided(keep, (T, N), (N + pad, 1), offset).fill_(False)
        assert (yb[keep] == 5.0).all()


@pytest.mark.parametrize("T,N", [(20, 256), (300, 256), (2500, 1024)])
def test_quantised_output_with_a_pitch(m, T, N):
    K = 272
    a = forward_inputs(T, N, K, 11)
    op = m.Fp8Linear(K, N, act="swiglu", quant="fp8", device=DEV)
    ref = op.forward(*a)
    o = op.buffers(T)
    wide = torch.full((T, N // 2 + 48), 9, dtype=torch.uint8, device=DEV)
    o.codes = wide[:, 16:16 + N // 2]
    op.forward(*a, out=o)
    assert torch.equal(o.codes, ref.codes) and torch.equal(o.sf, ref.sf)
    assert (wide[:, :16] == 9).all() and (wide[:, 16 + N // 2:] == 9).all()


@pytest.mark.parametrize("T,N,K", [(5, 144, 400), (40, 144, 400), (200, 272, 400), (2500, 1040, 272)])
def test_zero_scales_nan_codes_and_infinities_stay_in_their_rows(m, T, N, K):
    x, x_sf, w, w_sf = forward_inputs(T, N, K, 4)
    op = m.Fp8Linear(K, N, out_dtype=F32, device=DEV)
    clean = op.forward(x, x_sf, w, w_sf)
    x, x_sf = x.clone(), x_sf.clone()
    x_sf[1] = 0.0                  # an all-zero row
    x[2, 200] = 0x7F               # a NaN
    x_sf[3, 1] = math.inf
    x_sf[4] *= 2.0 ** -140         # subnormal
    out = op.forward(x, x_sf, w, w_sf)
    assert (out[1] == 0).all() and torch.isnan(out[2]).all() and not torch.isfinite(out[3]).any()
    y, err = ref_forward(x[4:5], x_sf[4:5], w, w_sf)
    assert ((out[4].double() - y[0]).abs() <= err[0] + 400 * 2.0 ** -149 * 448 * 448).all()
    keep = [0] + list(range(5, T))
    assert torch.equal(out[keep], clean[keep])


def test_swiglu_codes_of_zero_and_nan_rows(m):
    for T in (20, 300):
        x, x_sf, w, w_sf = forward_inputs(T, 512, 272, 8)
        x_sf[1] = 0.0
        x[2, 5] = 0x7F
        x_sf[3] *= 2.0 ** -40      # outputs of 2^-80 and less; below 2^-100 among them
        x_sf[4] *= 2.0 ** -52
        o = m.Fp8Linear(272, 512, act="swiglu", quant="fp8", device=DEV).forward(x, x_sf, w, w_sf)
        assert (o.sf[1] == 0).all() and ((o.codes[1] & 127) == 0).all()
        assert ((o.codes[2] & 127) == 127).all()
        y, err = swiglu(*ref_forward(x[3:5], x_sf[3:5], w, w_sf))
        err = err + 2.0 ** -149
        q = o.codes[3:5].view(torch.float8_e4m3fn).double() * o.sf[3:5].double().repeat_interleave(128, 1)
        assert ((q - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -9 * o.sf[3:5].double().repeat_interleave(128, 1) + 4 * err).all()


def test_no_tokens(m):
    op = m.Fp8Linear(144, 272, device=DEV)
    none = torch.empty(0, 144, dtype=torch.uint8, device=DEV)
    w, w_sf = random_codes(272, 144, 128, 128, 0)
    assert op.forward(none, torch.empty(0, 2, device=DEV), w, w_sf).shape == (0, 272)
    glu = m.Fp8Linear(144, 256, act="swiglu", quant="fp8", device=DEV)
    assert glu.forward(none, torch.empty(0, 2, device=DEV), w[:256], w_sf[:2]).sf.shape == (0, 1)
    dy = torch.empty(0, 272, dtype=torch.uint8, device=DEV)
    assert op.backward_input(dy, torch.empty(0, 3, device=DEV), w, w_sf).shape == (0, 144)
    args = (dy, torch.empty(0, 272, device=DEV), none, torch.empty(0, 144, device=DEV))
    out = torch.full((272, 144), 7.0, device=DEV)
    assert (op.backward_weight(*args, out=out) == 0).all()
    add = torch.randn(272, 144, device=DEV)
    assert torch.equal(op.backward_weight(*args, add=add, out=out), add)
    assert torch.equal(op.backward_weight(*args, add=add, out=add), out)


@pytest.mark.parametrize("T,N,K,rows", [(300001, 16, 7168, [0, 149799, 149800, 299593, 299594, 300000]),
                                        (40000, 65552, 16, [0, 1, 32759, 32760, 39999])])
def test_past_2_31_elements(m, T, N, K, rows):
    """Offsets of x, and of y, beyond 32 bits."""
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randint(0, 120, (T, K), generator=g, device=DEV, dtype=torch.uint8)
    x_sf = torch.rand(T, up(K), generator=g, device=DEV)
    w, w_sf = random_codes(N, K, 128, 128, 1)
    out = m.Fp8Linear(K, N, device=DEV).forward(x, x_sf, w, w_sf)
    y, err = ref_forward(x[rows], x_sf[rows], w, w_sf)
    close(out[rows], y, err)


def test_weight_gradient_past_2_31_elements(m):
    T, N, K = 20, 65552, 32784
    dy, dy_sf = random_codes(T, N, 128, 1, 0)
    x, x_sf = random_codes(T, K, 128, 1, 1)
    rows = [0, 1, 65503, 65504, 65505, N - 1]
    dw = m.Fp8Linear(K, N, device=DEV).backward_weight(dy, dy_sf, x, x_sf)
    ref, err = product(values(dy, dy_sf, 128, 1).t()[rows], values(x, x_sf, 128, 1).t(), 1)
    close(dw[rows], ref, err)


@pytest.mark.parametrize("T,N,K", [(40, 272, 144), (2500, 1040, 272)])
def test_gradients_against_differences(m, T, N, K):
    """The loss sum(dy y) is linear in a scale of x or W: its exact difference quotient is the sum of the gradient over the group,
    weighted by the codes.  y, dx and dw are f32 and their errors those of their sums."""
    x, x_sf, w, w_sf = forward_inputs(T, N, K, 9)
    op = m.Fp8Linear(K, N, out_dtype=F32, device=DEV)
    dy, dy_sf = random_codes(T, N, 1, 128, 2)
    d = values(dy, dy_sf, 1, 128)
    y = op.forward(x, x_sf, w, w_sf).double()
    dx = op.backward_input(dy, dy_sf, w, w_sf).double()
    X, W = values(x, x_sf, 1, 128), values(w, w_sf, 128, 128)
    mags = d.abs() @ W.abs()
    for t, b in ((0, 0), (T // 2, up(K) - 1), (T - 1, 0)):
        s = x_sf.clone()
        s[t, b] *= 2
        diff = (d[t] * (op.forward(x, s, w, w_sf).double()[t] - y[t])).sum()
        grad = (X[t, 128 * b:128 * b + 128] * dx[t, 128 * b:128 * b + 128]).sum()
        tol = 3 * 2.0 ** -15 * (X[t].abs() * mags[t]).sum()
        assert (diff - grad).abs() <= tol
    # the weight's: the same numbers with scales along the tokens (powers of two alone change nothing in the values)
    s1, s2 = 2.0 ** -3, 2.0 ** 2
    one = lambda t, v: torch.full((up(T), t.shape[1]), v, device=DEV)  # noqa: E731
    dw = op.backward_weight(dy, one(dy, s1), x, one(x, s2)).double()
    D, Xc = values(dy, one(dy, s1), 128, 1), values(x, one(x, s2), 128, 1)
    for i, j in ((0, 0), (up(N) - 1, up(K) - 1)):
        s = w_sf.clone()
        s[i, j] *= 2
        flat = torch.full_like(x_sf, s2)
        diff = (D * (op.forward(x, flat, w, s).double() - op.forward(x, flat, w, w_sf).double())).sum()
        blk = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
        grad = (W[blk] * dw[blk]).sum()
        tol = 3 * 2.0 ** -15 * (W.abs() * (D.abs().t() @ Xc.abs())).sum()
        assert (diff - grad).abs() <= tol


@pytest.mark.parametrize("T", [1, 40, 300, 3000])
def test_repeats_streams_and_capture(m, T):
    N, K = 1024, 1040
    a = forward_inputs(T, N, K, 6)
    op = m.Fp8Linear(K, N, act="swiglu", quant="fp8", device=DEV)
    dy, dy_sf = random_codes(T, N, 1, 128, 2)
    col, col_sf = random_codes(T, N, 128, 1, 2)
    xc, xc_sf = random_codes(T, K, 128, 1, 3)

    def everything(out=(None, None, None), stream=None):
        o = op.forward(*a, out=out[0], stream=stream)
        return o, op.backward_input(dy, dy_sf, a[2], a[3], out=out[1], stream=stream), op.backward_weight(col, col_sf, xc, xc_sf, out=out[2], stream=stream)

    flat = lambda r: (r[0].codes, r[0].sf, r[1], r[2])  # noqa: E731
    first = [t.clone() for t in flat(everything())]
    assert all(torch.equal(p, q) for p, q in zip(first, flat(everything())))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = everything(stream=s)
    here = everything()              # on two streams at once: nothing is shared
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(first, flat(side), flat(here)))
    out = op.buffers(T), op.input_grad_buffer(T), op.weight_grad_buffer()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        everything(out)
        with torch.cuda.graph(g, stream=s):
            everything(out)
    for t in flat(out):
        t.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, flat(out)))


@pytest.mark.parametrize("T,N,K", [(20, 272, 400), (300, 272, 400), (2500, 1040, 400)])
def test_a_wait_that_runs_out(m, T, N, K):
    """CTA 0 withholds its copies for one call: its waits give up, the status says so once, the next call is as before."""
    a = forward_inputs(T, N, K, 13)
    op = m.Fp8Linear(K, N, device=DEV)
    before = op.forward(*a)
    torch.cuda.synchronize()
    assert m.lib().moe_fp8_linear_status() == m.MOE_OK
    assert m.lib().moe_fp8_linear_test_arm_timeout(0) == m.MOE_ERR_INVALID_ARG
    assert m.lib().moe_fp8_linear_test_arm_timeout(20000) == m.MOE_OK
    op.forward(*a)
    assert m.lib().moe_fp8_linear_status() == m.MOE_ERR_DEVICE_TIMEOUT
    assert m.lib().moe_fp8_linear_status() == m.MOE_OK
    assert torch.equal(op.forward(*a), before)
    assert m.lib().moe_fp8_linear_status() == m.MOE_OK
