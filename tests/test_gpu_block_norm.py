"""BlockNorm against the formulas in 64 bits: shapes, types, pitches, masked
and degenerate rows, both quantised formats, gradients against the formula and
against differences.

Tolerances.  An output is one rounding of an f32 value: half a unit in the
last place, 2^-9 (bf16) or 2^-24 (f32) of the value, doubled where the f32
value falls on the other side of a rounding boundary.  The f32 value itself
carries a handful of roundings of terms whose magnitudes `mag` bounds, and
sums of a tree or a short chain: 2^-20 of `mag` covers 16 roundings.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def close(got, ref, what, mag=None):
    """Elementwise bound of the module's docstring; non-finite values must agree in kind."""
    got64, ref = got.detach().double().cpu(), ref.double().cpu()
    assert got64.shape == ref.shape, what
    u = 2.0 ** -8 if got.dtype == BF else 2.0 ** -20
    finite = torch.isfinite(ref)
    assert torch.equal(finite, torch.isfinite(got64)), f"{what}: non-finite values differ"
    mag = ref.abs() if mag is None else mag.double().cpu().expand_as(ref)
    tol = u * ref.abs() + 2.0 ** -20 * mag + 1e-37
    err = (got64 - ref).abs()
    bad = finite & ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {ref.numel()} off, worst {float((err / tol)[finite].max()):.3g} x tolerance"


def pitched(x, pad, offset):
    """The same values with `pad` extra elements per row and the first element `offset` into the allocation."""
    T, H = x.shape
    buf = torch.full((T * (H + pad) + offset + 8,), 77.0, dtype=x.dtype, device=x.device)
    v = torch.as_strided(buf, (T, H), (H + pad, 1), offset)
    v.copy_(x)
    return v


def make(T, H, dtype, pdtype, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    d = {"residual": r(T, H).to(dtype), "y": (0.5 * r(T, H)).to(dtype), "w_post": (1 + 0.2 * r(H)).to(pdtype),
         "w_pre": (1 + 0.2 * r(H)).to(pdtype), "dh": r(T, H).to(dtype), "dn": r(T, H).to(dtype), "gate": None}
    if gate:
        d["gate"] = r(H if gate == "channel" else T).to(pdtype)
    return {n: None if t is None else t.to(DEV) for n, t in d.items()}


def ref_forward(d, rs, gate, y=True, post=True, pre=True):
    f = {n: t.double().cpu() for n, t in d.items() if t is not None}
    o, z, u, mag = {}, f["residual"], None, f["residual"].abs()
    H = z.shape[1]
    if y:
        u = f["y"]
        if post:
            o["r1"] = (u.pow(2).sum(1) / H + EPS).rsqrt()
            u = u * o["r1"][:, None] * f["w_post"]
        gt = 1.0 if d["gate"] is None else f["gate"] if gate == "channel" else f["gate"][:, None]
        z = rs * f["residual"] + gt * u
        mag = abs(rs) * f["residual"].abs() + (gt * u).abs()
    o["h"], o["mag"] = z, mag
    if pre:
        o["r2"] = (z.pow(2).sum(1) / H + EPS).rsqrt()
        o["n"] = z * o["r2"][:, None] * f["w_pre"]
        o["nmag"] = mag * o["r2"][:, None] * f["w_pre"].abs()
    return o


def ref_backward(d, o, rs, gate, y=True, post=True, pre=True, dh=True):
    f = {n: t.double().cpu() for n, t in d.items() if t is not None}
    g = {}
    D = f["dh"] if dh else torch.zeros_like(f["residual"])
    if pre:
        a, hat = f["dn"] * f["w_pre"], o["h"] * o["r2"][:, None]
        g["dw_pre"], g["dw_pre_mag"] = (f["dn"] * hat).sum(0), (f["dn"] * hat).abs().sum(0)
        D = D + o["r2"][:, None] * (a - hat * (a * hat).mean(1, keepdim=True))
    g["dresidual"] = D * (rs if y else 1.0)
    if y:
        gt = 1.0 if d["gate"] is None else f["gate"] if gate == "channel" else f["gate"][:, None]
        u, inner = f["y"], D * gt
        if post:
            hat = f["y"] * o["r1"][:, None]
            u = hat * f["w_post"]
            g["dw_post"], g["dw_post_mag"] = (inner * hat).sum(0), (inner * hat).abs().sum(0)
            b = inner * f["w_post"]
            g["dy"] = o["r1"][:, None] * (b - hat * (b * hat).mean(1, keepdim=True))
        else:
            g["dy"] = inner
        if d["gate"] is not None:
            dim = 0 if gate == "channel" else 1
            g["dgate"], g["dgate_mag"] = (D * u).sum(dim), (D * u).abs().sum(dim)
    return g


SHAPES = [(1, 1), (2, 7), (3, 32), (5, 96), (1, 128), (4, 129), (7, 1000), (3, 1001), (2, 2056), (5, 4096), (33, 7168),
          (3, 8320), (2, 14336), (2, 16384)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)], ids=["bf16", "bf16_bf16", "f32", "f32_bf16"])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_forward_matches_formula(m, T, H, dtype, pdtype, gate):
    d = make(T, H, dtype, pdtype, gate, seed=T * 31 + H)
    op = m.BlockNorm(H, EPS, residual_scale=0.75, gate=gate, dtype=dtype, param_dtype=pdtype, device=DEV)
    out = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"])
    ref = ref_forward(d, 0.75, gate)
    close(out.h, ref["h"], "h", ref["mag"])
    close(out.n, ref["n"], "n", ref["nmag"])
    close(out.rstd_post, ref["r1"], "rstd_post")
    close(out.rstd_pre, ref["r2"], "rstd_pre")


@pytest.mark.parametrize("y,post,pre", [(True, True, False), (True, False, True), (True, False, False), (False, False, True)])
@pytest.mark.parametrize("H", [129, 1024])
def test_forward_parts(m, y, post, pre, H):
    T = 6
    d = make(T, H, BF, F32, "channel" if y else None, seed=5)
    op = m.BlockNorm(H, EPS, residual_scale=0.5, gate="channel" if y else None, device=DEV)
    out = op.forward(d["residual"], d["y"] if y else None, d["w_post"] if post else None, d["gate"], d["w_pre"] if pre else None)
    ref = ref_forward(d, 0.5, "channel", y, post, pre)
    if y:
        close(out.h, ref["h"], "h", ref["mag"])
    else:
        assert out.h is None
    if pre:
        close(out.n, ref["n"], "n", ref["nmag"])


def check_codes(codes, sf, v, quant):
    """Codes are within half an E4M3 step of v / sf, scales are the format's."""
    G = 128 if quant == "fp8" else 32
    T, H = v.shape
    top = v.view(T, H // G, G).abs().amax(2)
    if quant == "fp8":
        close(sf, top / 448, "sf")
        s = sf.double().cpu()
    else:
        e = sf.cpu().to(torch.int32) - 127
        exact = torch.ceil(torch.log2(top / 448)).clamp(-127, 127)
        exact = torch.where(top > 0, exact, torch.full_like(exact, -127.0))
        # a ratio within f32 rounding of a power of two may round onto it
        near = (torch.log2(top / 448) - torch.round(torch.log2(top / 448))).abs() < 2.0 ** -18
        assert ((e == exact) | (near & ((e - exact).abs() <= 1))).all(), "UE8M0 scales"
        s = torch.ldexp(torch.ones(()).double(), e.double())
    s = s.repeat_interleave(G, 1)
    q = codes.view(torch.float8_e4m3fn).float().cpu().double()
    # saturation never bites: |v| / sf <= 448 up to rounding
    tol = (2.0 ** -4 * v.abs() + 2.0 ** -10 * s) * (1 + 2.0 ** -16)
    bad = (q * s - v).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} codes off"


@pytest.mark.parametrize("quant,H", [("fp8", 128), ("fp8", 1152), ("fp8", 7168), ("fp8", 16384), ("ue8m0", 32), ("ue8m0", 160),
                                     ("ue8m0", 4096), ("ue8m0", 7168)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_quantised_outputs(m, quant, H, dtype):
    T = 9
    d = make(T, H, dtype, F32, "token", seed=H)
    d["residual"][3] = 0
    d["y"][3] = 0                                   # a padding row: zero groups, scale 0, codes 0
    d["residual"][4] *= 1e-18                       # tiny and huge rows normalise all the same
    d["y"][4] *= 1e-18
    d["residual"][5] *= 1e15
    op = m.BlockNorm(H, EPS, gate="token", quant=quant, dtype=dtype, device=DEV)
    for normed in (True, False):
        out = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"], normed=normed)
        ref = ref_forward(d, 1.0, "token")
        close(out.h, ref["h"], "h", ref["mag"])
        assert (out.n is None) == (not normed)
        if normed:
            close(out.n, ref["n"], "n", ref["nmag"])
        check_codes(out.codes, out.sf, ref["n"], quant)
        assert (out.codes[3] == 0).all() and (out.sf[3] == 0).all()


def test_quantised_input_feeds_the_layer(m):
    """codes and sf are what MoELayer.forward takes: y of the layer on them against y on the same values quantised by
    the synthetic inputs' recipe."""
    import moe_synth
    wl = moe_synth.WORKLOADS["tiny"]
    inp = {n: t.to(DEV) for n, t in moe_synth.make_inputs(wl).items()}
    layer = m.MoELayer(wl.T, wl.H, wl.I, wl.E, wl.k, device=DEV)
    layer.transform_weights(inp["w1"], inp["w1_sf"], inp["w2"], inp["w2_sf"])
    d = make(wl.T, wl.H, BF, F32, None, seed=3)
    op = m.BlockNorm(wl.H, EPS, quant="fp8", device=DEV)
    out = op.forward(d["residual"], w_pre=d["w_pre"])
    v = ref_forward(d, 1.0, None, y=False)["n"].float()
    q, sf = moe_synth.pack_fp8_rows_f32(v)
    a = layer.forward(out.codes, out.sf, inp["topk_idx"], inp["topk_weights"]).float()
    b = layer.forward(q.to(DEV), sf.to(DEV), inp["topk_idx"], inp["topk_weights"]).float()
    # the two inputs may differ in a code on a rounding boundary here and there: 1 code in 1000 by 2^-3 is 4e-3
    assert (a - b).norm() <= 4e-3 * b.norm()


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (8, 0), (3, 5), (16, 8)])
@pytest.mark.parametrize("H", [256, 1000])
def test_pitches_and_alignment(m, pad, offset, H):
    T = 5
    d = make(T, H, BF, F32, "channel", seed=9)
    op = m.BlockNorm(H, EPS, gate="channel", device=DEV)
    want = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"])
    out = op.buffers(T)
    out.h, out.n = pitched(torch.zeros(T, H, dtype=BF, device=DEV), pad, offset), pitched(torch.zeros(T, H, dtype=BF, device=DEV), pad + 2, offset)
    hbase, nbase = out.h._base if out.h._base is not None else out.h, out.n._base if out.n._base is not None else out.n
    before = hbase.clone(), nbase.clone()
    op.forward(pitched(d["residual"], pad, offset), pitched(d["y"], pad + 1, offset), d["w_post"], d["gate"], d["w_pre"], out=out)
    ref = ref_forward(d, 1.0, "channel")
    close(out.h, ref["h"], "h", ref["mag"])
    close(out.n, ref["n"], "n", ref["nmag"])
    close(out.rstd_pre, want.rstd_pre, "rstd_pre")
    # nothing was written outside the rows
    for base, old, v in ((hbase, before[0], out.h), (nbase, before[1], out.n)):
        keep = torch.ones_like(base, dtype=torch.bool)
        torch.as_strided(keep, v.shape, v.stride(), v.storage_offset()).fill_(False)
        assert torch.equal(base[keep], old[keep])
    g0 = op.backward(d["residual"], d["dh"], d["dn"], d["y"], d["w_post"], d["gate"], d["w_pre"], want.rstd_post, want.rstd_pre)
    gr = op.grad_buffers(T)
    gr.dresidual, gr.dy = pitched(torch.zeros(T, H, dtype=BF, device=DEV), pad, offset), pitched(torch.zeros(T, H, dtype=BF, device=DEV), pad, offset)
    op.backward(pitched(d["residual"], pad, offset), pitched(d["dh"], pad, offset), pitched(d["dn"], pad + 1, offset), pitched(d["y"], pad, offset),
                d["w_post"], d["gate"], d["w_pre"], want.rstd_post, want.rstd_pre, out=gr)
    for name in ("dresidual", "dy", "dw_post", "dgate", "dw_pre"):
        a, b = getattr(g0, name).double(), getattr(gr, name).double()
        # the same f32 terms, summed in another order where the pitches call for another access width
        assert (a - b).abs().max() <= (2.0 ** -7 if getattr(g0, name).dtype == BF else 2.0 ** -16) * a.abs().max(), name


def test_in_place_stream(m):
    """h may be the residual itself, dresidual dh, dy dn."""
    T, H = 37, 1152
    d = make(T, H, BF, F32, "channel", seed=21)
    op = m.BlockNorm(H, EPS, gate="channel", quant="fp8", device=DEV)
    want = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"])
    out = op.buffers(T)
    out.h = d["residual"].clone()
    op.forward(out.h, d["y"], d["w_post"], d["gate"], d["w_pre"], out=out)
    for n in ("h", "n", "codes", "sf", "rstd_post", "rstd_pre"):
        assert torch.equal(getattr(out, n), getattr(want, n)), n
    args = (d["y"], d["w_post"], d["gate"], d["w_pre"], want.rstd_post, want.rstd_pre)
    g = op.backward(want.h, d["dh"], d["dn"], *args)
    g2 = op.grad_buffers(T)
    g2.dresidual, g2.dy = d["dh"].clone(), d["dn"].clone()
    op.backward(want.h, g2.dresidual, g2.dy, *args, out=g2)
    for n in ("dresidual", "dy", "dw_post", "dgate", "dw_pre"):
        assert torch.equal(getattr(g, n), getattr(g2, n)), n


@pytest.mark.parametrize("H", [96, 1024, 1001])
def test_non_finite_rows_stay_in_their_rows(m, H):
    """A row with a NaN or an infinity is NaN where the formula is; its neighbours are untouched."""
    T = 6
    d = make(T, H, F32, F32, None, seed=2)
    op = m.BlockNorm(H, EPS, dtype=F32, device=DEV)
    clean = op.forward(d["residual"], d["y"], d["w_post"], None, d["w_pre"])
    d["y"][1, H // 2] = math.nan
    d["residual"][4, 0] = math.inf
    out = op.forward(d["residual"], d["y"], d["w_post"], None, d["w_pre"])
    keep = [0, 2, 3, 5]
    assert torch.equal(out.n[keep], clean.n[keep]) and torch.equal(out.h[keep], clean.h[keep])
    assert torch.isnan(out.h[1]).all() and torch.isnan(out.n[1]).all()
    assert torch.isinf(out.h[4, 0]) and torch.isnan(out.n[4, 0]) and (out.n[4, 1:] == 0).all()


def test_zero_rows(m):
    """All-zero rows (padding): eps keeps the reciprocal roots finite, outputs and gradients are finite."""
    T, H = 3, 256
    z = torch.zeros(T, H, dtype=BF, device=DEV)
    one = torch.ones(H, device=DEV)
    op = m.BlockNorm(H, EPS, device=DEV)
    out = op.forward(z, z, one, None, one)
    assert (out.h == 0).all() and (out.n == 0).all()
    assert torch.allclose(out.rstd_pre, torch.full((T,), 1000.0, device=DEV), rtol=1e-5)
    g = op.backward(out.h, torch.ones_like(z), torch.ones_like(z), z, one, None, one, out.rstd_post, out.rstd_pre)
    for n in ("dresidual", "dy", "dw_post", "dw_pre"):
        assert torch.isfinite(getattr(g, n).float()).all(), n
    assert torch.allclose(g.dresidual.float(), torch.full((T, H), 1001.0, device=DEV), rtol=2.0 ** -8)


def test_no_tokens(m):
    H = 384
    op = m.BlockNorm(H, EPS, gate="channel", quant="fp8", device=DEV)
    e = torch.empty(0, H, dtype=BF, device=DEV)
    p = torch.ones(H, device=DEV)
    out = op.forward(e, e, p, p, p)
    assert out.h.shape == (0, H) and out.codes.shape == (0, H)
    g = op.grad_buffers(0)
    g.dw_post.fill_(3)
    g.dgate.fill_(3)
    g.dw_pre.fill_(3)
    r = torch.empty(0, device=DEV)
    op.backward(e, e, e, e, p, p, p, r, r, out=g)
    assert (g.dw_post == 0).all() and (g.dgate == 0).all() and (g.dw_pre == 0).all()


@pytest.mark.parametrize("T,H", [(1, 1), (2, 33), (3, 128), (700, 136), (5, 1000), (401, 1001), (33, 7168), (3, 14336), (2, 16384)])
@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (F32, F32), (BF, BF)], ids=["bf16", "f32", "bf16_bf16"])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_backward_matches_formula(m, T, H, dtype, pdtype, gate):
    d = make(T, H, dtype, pdtype, gate, seed=T + 3 * H)
    op = m.BlockNorm(H, EPS, residual_scale=0.75, gate=gate, dtype=dtype, param_dtype=pdtype, device=DEV)
    fwd = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"])
    g = op.backward(fwd.h, d["dh"], d["dn"], d["y"], d["w_post"], d["gate"], d["w_pre"], fwd.rstd_post, fwd.rstd_pre)
    o = {"h": fwd.h.double().cpu(), "r1": fwd.rstd_post.double().cpu(), "r2": fwd.rstd_pre.double().cpu()}
    ref = ref_backward(d, o, 0.75, gate)
    # D and dy are differences of terms of about the size of dh + r2 dn w_pre (a row's largest bounds them)
    D = ref["dresidual"] / 0.75
    big = (d["dh"].double().cpu().abs() + o["r2"][:, None] * (d["dn"].double().cpu() * d["w_pre"].double().cpu()).abs()).amax(1, keepdim=True)
    wide = 4 * big * (1 + (o["h"] * o["r2"][:, None]).abs())
    close(g.dresidual, ref["dresidual"], "dresidual", wide)
    gmax = 1.0 if d["gate"] is None else d["gate"].double().cpu().abs().max()
    hat = (d["y"].double().cpu() * o["r1"][:, None]).abs()
    close(g.dy, ref["dy"], "dy", 8 * wide.amax(1, keepdim=True) * gmax * o["r1"][:, None] * 2 * (1 + hat))
    # sums over tokens of products of D: D's own error is 2^-20 of `wide` per term
    for n in ("dw_pre", "dw_post", "dgate"):
        if n not in ref:
            assert getattr(g, n) is None
            continue
        slack = ref[n + "_mag"]
        if n != "dw_pre":
            axis = 1 if (n == "dgate" and gate == "token") else 0
            slack = slack + (wide * hat * 2 * (gmax if n == "dw_post" else 1.0)).sum(axis)
        close(getattr(g, n), ref[n], n, slack)
    assert torch.isfinite(D).all()


@pytest.mark.parametrize("y,post,pre,dh", [(True, True, False, True), (True, False, True, True), (True, True, True, False),
                                           (False, False, True, True), (False, False, True, False)])
def test_backward_parts(m, y, post, pre, dh):
    T, H = 19, 264
    gate = "channel" if y else None
    d = make(T, H, F32, F32, gate, seed=8)
    op = m.BlockNorm(H, EPS, residual_scale=2.0, gate=gate, dtype=F32, device=DEV)
    args = (d["y"] if y else None, d["w_post"] if post else None, d["gate"], d["w_pre"] if pre else None)
    fwd = op.forward(d["residual"], *args) if y or pre else None
    h = fwd.h if y else d["residual"]
    g = op.backward(h, d["dh"] if dh else None, d["dn"] if pre else None, *args, fwd.rstd_post, fwd.rstd_pre)
    o = {"h": h.double().cpu(), "r1": None if fwd.rstd_post is None else fwd.rstd_post.double().cpu(),
         "r2": None if fwd.rstd_pre is None else fwd.rstd_pre.double().cpu()}
    ref = ref_backward(d, o, 2.0, gate, y, post, pre, dh)
    for n in ("dresidual", "dy", "dw_post", "dgate", "dw_pre"):
        if n in ref:
            # f32 throughout: 2^-16 of the largest is far above the roundings and far below a wrong term
            assert (getattr(g, n).double().cpu() - ref[n]).abs().max() <= 2.0 ** -16 * ref[n].abs().max(), n


@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("H", [40, 129])
def test_backward_against_differences(m, gate, H):
    """Directional derivative of sum(h dh + n dn) by central differences of the forward kernel.  Step 2^-7 leaves a
    truncation error of about step^2, the f32 forward one of 2^-24 / 2^-7 of the sum's terms: 2^-10 of the scale."""
    T = 4
    d = make(T, H, F32, F32, gate, seed=H)
    op = m.BlockNorm(H, EPS, residual_scale=0.5, gate=gate, dtype=F32, device=DEV)

    def loss(v):
        o = op.forward(v["residual"], v["y"], v["w_post"], v["gate"], v["w_pre"])
        return float((o.h.double() * d["dh"].double()).sum() + (o.n.double() * d["dn"].double()).sum())

    fwd = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"])
    g = op.backward(fwd.h, d["dh"], d["dn"], d["y"], d["w_post"], d["gate"], d["w_pre"], fwd.rstd_post, fwd.rstd_pre)
    grads = {"residual": g.dresidual, "y": g.dy, "w_post": g.dw_post, "w_pre": g.dw_pre, "gate": g.dgate}
    step = 2.0 ** -7
    gen = torch.Generator().manual_seed(1)
    for n, gr in grads.items():
        if gr is None:
            continue
        v = torch.randn(d[n].shape, generator=gen).to(DEV)
        up, dn = ({**d, n: d[n] + s * step * v} for s in (1, -1))
        num = (loss(up) - loss(dn)) / (2 * step)
        ana = float((gr.double() * v.double()).sum())
        scale = float((gr.double() * v.double()).abs().sum())
        assert abs(num - ana) <= 2.0 ** -10 * scale, (n, num, ana, scale)


def test_repeatable_and_on_another_stream(m):
    T, H = 997, 1288
    d = make(T, H, BF, F32, "channel", seed=4)
    op = m.BlockNorm(H, EPS, gate="channel", device=DEV)
    fwd = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"])
    args = (fwd.h, d["dh"], d["dn"], d["y"], d["w_post"], d["gate"], d["w_pre"], fwd.rstd_post, fwd.rstd_pre)
    a = op.backward(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = op.backward(*args, stream=side)
    f2 = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"], stream=side)
    side.synchronize()
    for n in ("dresidual", "dy", "dw_post", "dgate", "dw_pre"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    assert torch.equal(fwd.h, f2.h) and torch.equal(fwd.n, f2.n)


def test_graph_capture(m):
    T, H = 17, 896
    d = make(T, H, BF, F32, "token", seed=6)
    op = m.BlockNorm(H, EPS, gate="token", quant="ue8m0", device=DEV)
    out, eager = op.buffers(T), op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"], out=out)
        with torch.cuda.graph(g, stream=s):
            op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"], out=out)
    out.h.zero_()
    out.codes.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.h, eager.h) and torch.equal(out.codes, eager.codes) and torch.equal(out.sf, eager.sf)


def test_offsets_past_32_bits(m):
    """A stream whose last rows start past 2^31 elements (a large pitch, few rows)."""
    T, H, pitch = 3, 1024, 1_100_000_003
    d = make(T, H, BF, F32, None, seed=12)
    big = torch.empty((T - 1) * pitch + H, dtype=BF, device=DEV)
    far = torch.as_strided(big, (T, H), (pitch, 1))
    far.copy_(d["residual"])
    op = m.BlockNorm(H, EPS, device=DEV)
    want = op.forward(d["residual"], d["y"], d["w_post"], None, d["w_pre"])
    out = op.buffers(T)
    out.h = far                                    # in place, far apart
    op.forward(far, d["y"], d["w_post"], None, d["w_pre"], out=out)
    ref = ref_forward(d, 1.0, None)
    close(out.h, ref["h"], "h", ref["mag"])
    close(out.n, ref["n"], "n", ref["nmag"])
    assert torch.equal(out.rstd_post, want.rstd_post) or torch.allclose(out.rstd_post, want.rstd_post, rtol=1e-6)


@pytest.mark.parametrize("T,H", [(161, 1024), (400, 776), (310, 520), (700, 5000)])
@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (F32, BF)], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_forward_of_many_rows(m, T, H, dtype, pdtype, gate):
    """More rows than SMs: CTAs that walk rows."""
    test_forward_matches_formula(m, T, H, dtype, pdtype, gate)


@pytest.mark.parametrize("quant,H", [("fp8", 640), ("fp8", 1024), ("ue8m0", 544), ("ue8m0", 992), ("fp8", 2048)])
@pytest.mark.parametrize("T", [1, 200])
def test_quantised_outputs_of_short_rows(m, quant, H, T):
    d = make(T, H, BF, F32, "token", seed=T + H)
    op = m.BlockNorm(H, EPS, gate="token", quant=quant, device=DEV)
    out = op.forward(d["residual"], d["y"], d["w_post"], d["gate"], d["w_pre"])
    ref = ref_forward(d, 1.0, "token")
    close(out.h, ref["h"], "h", ref["mag"])
    close(out.n, ref["n"], "n", ref["nmag"])
    check_codes(out.codes, out.sf, ref["n"], quant)


@pytest.mark.parametrize("T,H", [(2432, 1024), (2701, 264), (4870, 8), (1217, 1288), (1900, 2048)])
@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (F32, F32), (F32, BF)], ids=["bf16", "f32", "f32_bf16"])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_backward_of_many_short_rows(m, T, H, dtype, pdtype, gate):
    """Several CTAs an SM, each with rows for two passes and more."""
    test_backward_matches_formula(m, T, H, dtype, pdtype, gate)


@pytest.mark.parametrize("T,H", [(5, 2501), (161, 4001), (310, 4097), (4, 8191), (3, 9001), (700, 4096), (460, 2560), (301, 8200)])
@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (F32, BF)], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_wide_rows_by_element_and_several_ctas_an_sm(m, T, H, dtype, pdtype, gate):
    test_forward_matches_formula(m, T, H, dtype, pdtype, gate)
    test_backward_matches_formula(m, T, H, dtype, pdtype, gate)
