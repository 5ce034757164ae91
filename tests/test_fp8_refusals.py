"""Argument checks of the FP8 linear and quantiser and of the router's groups: made on the host before anything is launched, so
they need no GPU."""
import math
import warnings

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


BAD = -1
P = 1 << 20        # stands for an aligned device pointer; never dereferenced by a refused call
CPU = torch.device("cpu")
U8, BF = torch.uint8, torch.bfloat16


def lcfg(m, **kw):
    return m.Fp8LinearConfig(*{**dict(in_features=256, out_features=512, act=0, quant=0, out_dtype=0, act_clamp=math.inf), **kw}.values())


BAD_LINEAR = [dict(in_features=0), dict(in_features=8), dict(in_features=264), dict(in_features=-16), dict(in_features=(1 << 20) + 16),
              dict(out_features=0), dict(out_features=24), dict(out_features=(1 << 20) + 16), dict(act=2), dict(act=1, out_features=128),
              dict(act=1, out_features=384), dict(quant=1), dict(quant=2, act=1), dict(quant=-1), dict(out_dtype=2), dict(act_clamp=0.0),
              dict(act_clamp=-1.0), dict(act_clamp=math.nan)]


def forward(m, c, T=4, x=P, ld_x=256, x_sf=P, w=P, w_sf=P, add=None, ld_add=0, y=P, ld_y=512, y_sf=None):
    return m.lib().moe_fp8_linear_forward(c, T, x, ld_x, x_sf, w, w_sf, add, ld_add, y, ld_y, y_sf, None)


def backward_input(m, c, T=4, dy=P, ld_dy=512, dy_sf=P, w=P, w_sf=P, add=None, ld_add=0, dx=P, ld_dx=256):
    return m.lib().moe_fp8_linear_backward_input(c, T, dy, ld_dy, dy_sf, w, w_sf, add, ld_add, dx, ld_dx, None)


def backward_weight(m, c, T=4, dy=P, ld_dy=512, dy_sf=P, x=P, ld_x=256, x_sf=P, add=None, ld_add=0, dw=P, ld_dw=256):
    return m.lib().moe_fp8_linear_backward_weight(c, T, dy, ld_dy, dy_sf, x, ld_x, x_sf, add, ld_add, dw, ld_dw, None)


@pytest.mark.parametrize("kw", BAD_LINEAR)
def test_linear_config(m, kw):
    for f in (forward, backward_input, backward_weight):
        assert f(m, lcfg(m, **kw)) == BAD and f(m, lcfg(m, **kw), T=0) == BAD
    assert forward(m, None) == BAD


def test_no_tokens_is_no_call(m):
    assert forward(m, lcfg(m), T=0, x=None, y=None) == 0 and backward_input(m, lcfg(m), T=0, dy=None, dx=None) == 0


@pytest.mark.parametrize("kw", [dict(T=-1), dict(x=None), dict(x=P + 8), dict(ld_x=255), dict(ld_x=264), dict(x_sf=None), dict(x_sf=P + 2),
                                dict(w=None), dict(w=P + 8), dict(w_sf=None), dict(w_sf=P + 1), dict(y=None), dict(y=P + 8), dict(ld_y=511),
                                dict(ld_y=513), dict(add=P, ld_add=511), dict(add=P, ld_add=514), dict(add=P + 2, ld_add=512), dict(y_sf=P)])
def test_forward(m, kw):
    assert forward(m, lcfg(m), **kw) == BAD


@pytest.mark.parametrize("kw", [dict(y_sf=None), dict(y_sf=P + 2), dict(y_sf=P, add=P, ld_add=256), dict(y_sf=P, ld_y=255), dict(y_sf=P, ld_y=264),
                                dict(y_sf=P, y=P + 4)])
def test_quantised_forward(m, kw):
    assert forward(m, lcfg(m, act=1, quant=1), **{**dict(ld_y=256), **kw}) == BAD


@pytest.mark.parametrize("kw", [dict(T=-1), dict(dy=None), dict(dy=P + 1), dict(ld_dy=511), dict(ld_dy=520), dict(dy_sf=None), dict(w=None),
                                dict(w_sf=None), dict(dx=None), dict(dx=P + 2), dict(ld_dx=255), dict(ld_dx=257), dict(add=P, ld_add=0)])
def test_backward_input(m, kw):
    assert backward_input(m, lcfg(m), **kw) == BAD


@pytest.mark.parametrize("kw", [dict(T=-1), dict(dy=None), dict(dy=P + 1), dict(ld_dy=511), dict(dy_sf=None), dict(dy_sf=P + 2), dict(x=None),
                                dict(x=P + 4), dict(ld_x=250), dict(x_sf=None), dict(dw=None), dict(dw=P + 4), dict(ld_dw=255), dict(ld_dw=257),
                                dict(add=P, ld_add=255), dict(add=P + 8, ld_add=256), dict(T=0, dw=None)])
def test_backward_weight(m, kw):
    assert backward_weight(m, lcfg(m), **kw) == BAD


def qcfg(m, **kw):
    return m.Fp8QuantConfig(*{**dict(columns=256, act=0, dtype=0, act_clamp=math.inf), **kw}.values())


OUT = dict(codes=P, sf=P, col_codes=P, col_sf=P)


@pytest.mark.parametrize("kw", [dict(columns=0), dict(columns=8), dict(columns=264), dict(columns=(1 << 20) + 16), dict(act=2), dict(act=1, columns=144),
                                dict(dtype=2), dict(act_clamp=0.0), dict(act_clamp=math.nan)])
def test_quant_config(m, kw):
    L, c = m.lib(), qcfg(m, **kw)
    assert L.moe_fp8_quant(c, 4, P, 4096, m.Fp8QuantIO(**OUT), None) == BAD and L.moe_fp8_quant(c, 0, None, 0, m.Fp8QuantIO(**OUT), None) == BAD
    assert L.moe_fp8_quant_weights(c, 4, P, 4096, P, P, None) == BAD
    assert L.moe_fp8_quant_backward(qcfg(m, **{**dict(act=1), **kw}), 4, P, 4096, P, 4096, m.Fp8QuantIO(**OUT), None) == BAD


@pytest.mark.parametrize("out", [dict(codes=None), dict(sf=None), dict(col_codes=None), dict(col_sf=None), dict(codes=P + 8), dict(col_codes=P + 4),
                                 dict(sf=P + 2), dict(col_sf=P + 8), dict(codes=None, sf=None, col_codes=None, col_sf=None)])
def test_quant_outputs(m, out):
    io = m.Fp8QuantIO(**{**OUT, **out})
    assert m.lib().moe_fp8_quant(qcfg(m), 4, P, 256, io, None) == BAD
    assert m.lib().moe_fp8_quant_backward(qcfg(m, act=1), 4, P, 256, P, 512, io, None) == BAD


def test_quant_inputs(m):
    L, io = m.lib(), m.Fp8QuantIO(**OUT)
    for T, v, ld in ((-1, P, 256), (4, None, 256), (4, P + 8, 256), (4, P, 255), (4, P, 257), (4, P, -256)):
        assert L.moe_fp8_quant(qcfg(m), T, v, ld, io, None) == BAD
        assert L.moe_fp8_quant_weights(qcfg(m), T, v, ld, P, P, None) == BAD
        assert L.moe_fp8_quant_backward(qcfg(m, act=1), T, v, ld, P, 512, io, None) == BAD
    assert L.moe_fp8_quant(qcfg(m, act=1), 4, P, 256, io, None) == BAD              # [T, 2H]
    assert L.moe_fp8_quant_backward(qcfg(m), 4, P, 256, P, 512, io, None) == BAD    # only of SwiGLU
    assert L.moe_fp8_quant_weights(qcfg(m, act=1), 4, P, 256, P, P, None) == BAD
    assert L.moe_fp8_quant_weights(qcfg(m), 4, P, 256, None, P, None) == BAD
    assert L.moe_fp8_quant_weights(qcfg(m), 4, P, 256, P, None, None) == BAD
    assert L.moe_fp8_quant(None, 4, P, 256, io, None) == BAD and L.moe_fp8_quant(qcfg(m), 4, P, 256, None, None) == BAD


def rcfg(m, **kw):
    d = dict(num_experts=64, topk=4, score=1, renormalize=1, logits_dtype=1, weight_scale=1.0, balance_coef=0.0, z_coef=0.0, bias_on=1, num_groups=8,
             topk_groups=4, group_score=0)
    return m.RouterConfig(*{**d, **kw}.values())


def test_groups(m):
    ok = lambda **kw: m.lib().moe_router_workspace_bytes(rcfg(m, **kw), 4, 1) > 0  # noqa: E731
    assert ok() and ok(topk_groups=8) and ok(topk_groups=1) and ok(group_score=1) and ok(num_groups=0, topk_groups=0)
    assert ok(num_experts=1024, num_groups=32) and ok(num_experts=32, num_groups=32, topk_groups=4)
    for kw in (dict(num_groups=1), dict(num_groups=-1), dict(num_groups=3), dict(num_groups=64), dict(topk_groups=0), dict(topk_groups=9),
               dict(topk_groups=-1), dict(group_score=2), dict(group_score=-1), dict(topk=9, topk_groups=1), dict(num_experts=1000, num_groups=25)):
        assert not ok(**kw), kw
    for kw in (dict(groups=0, topk_groups=1), dict(groups=8), dict(topk_groups=2)):
        with pytest.raises(ValueError, match="groups"):
            m.Router(64, 4, device=CPU, **kw)
    with pytest.raises(ValueError, match="group_score"):
        m.Router(64, 4, groups=8, topk_groups=2, group_score="sum", device=CPU)
    with pytest.raises(m.MoEError):
        m.Router(64, 4, groups=7, topk_groups=2, device=CPU)
    assert m.Router(64, 4, groups=8, topk_groups=2, device=CPU).cfg.num_groups == 8


def test_operators_of_bad_sizes(m):
    for make in (lambda: m.Fp8Linear(100, 128, device=CPU), lambda: m.Fp8Linear(128, 128, act="swiglu", device=CPU),
                 lambda: m.Fp8Linear(128, 128, quant="fp8", device=CPU), lambda: m.Fp8Linear(128, 256, act="swiglu", quant="ue8m0", device=CPU),
                 lambda: m.Fp8Quant(100, device=CPU), lambda: m.Fp8Quant(144, act="swiglu", device=CPU)):
        with pytest.raises(m.MoEError):
            make()
    for make, name in ((lambda: m.Fp8Linear(128, 128, act="gelu", device=CPU), "act"), (lambda: m.Fp8Linear(128, 128, out_dtype=torch.half, device=CPU), "dtype"),
                       (lambda: m.Fp8Quant(128, dtype=torch.half, device=CPU), "dtype")):
        with pytest.raises(ValueError, match=name):
            make()


def tensors(T=5, N=272, K=144):
    b = lambda n: (n + 127) // 128  # noqa: E731
    u8, f = (lambda *s: torch.zeros(*s, dtype=U8)), (lambda *s: torch.zeros(*s))
    return dict(x=u8(T, K), x_sf=f(T, b(K)), w=u8(N, K), w_sf=f(b(N), b(K)), dy=u8(T, N), dy_sf=f(T, b(N)), dyc_sf=f(b(T), N), xc_sf=f(b(T), K))


CHANGES = [lambda t: t[:-1], lambda t: t.double(), lambda t: t[0], lambda t: torch.zeros(t.shape[1], t.shape[0], dtype=t.dtype).t(), lambda t: "no tensor"]


def test_tensors_are_checked(m):
    op = m.Fp8Linear(144, 272, device=CPU)
    calls = {"forward": (("x", "x_sf", "w", "w_sf"), op.forward), "input": (("dy", "dy_sf", "w", "w_sf"), op.backward_input),
             "weight": (("dy", "dyc_sf", "x", "xc_sf"), op.backward_weight)}
    for names, call in calls.values():
        t = tensors()
        with pytest.raises(RuntimeError, match="CPU"):          # all in order: there is only no GPU
            call(*(t[n] for n in names))
        for i, n in enumerate(names):
            for change in CHANGES:
                bad = change(t[n])
                if isinstance(bad, torch.Tensor) and bad.shape == t[n].shape and bad.dtype == t[n].dtype and bad.is_contiguous():
                    continue
                args = [t[k] for k in names]
                args[i] = bad
                with pytest.raises((ValueError, TypeError, AttributeError, IndexError)):
                    call(*args)
        with pytest.raises((ValueError, TypeError)):
            call(*(t[n] for n in names), out=torch.zeros(1, 1))
        with pytest.raises((ValueError, TypeError)):
            call(*(t[n] for n in names), add=torch.zeros(1, 1))
    glu = m.Fp8Linear(144, 512, act="swiglu", quant="fp8", device=CPU)
    t = tensors(N=512)
    with pytest.raises(ValueError, match="add"):
        glu.forward(t["x"], t["x_sf"], t["w"], t["w_sf"], add=torch.zeros(5, 256, dtype=U8))


def test_quant_tensors_are_checked(m):
    op = m.Fp8Quant(256, act="swiglu", device=CPU)
    v, d = torch.zeros(5, 512, dtype=BF), torch.zeros(5, 256, dtype=BF)
    for call in (lambda: op.forward(v), lambda: op.backward(d, v), lambda: m.Fp8Quant(256, device=CPU).weights(d)):
        with pytest.raises(RuntimeError, match="CPU"):
            call()
    for call in (lambda: op.forward(d), lambda: op.forward(v.float()), lambda: op.backward(v, v), lambda: op.backward(d[:4], v),
                 lambda: op.backward(None, v), lambda: op.forward(v, out=op.buffers(4)), lambda: op.backward(d, v, out=op.buffers(5)),
                 lambda: m.Fp8Quant(256, device=CPU).weights(v)):
        with pytest.raises(ValueError):
            call()


def test_inputs_with_a_graph(m):
    t = tensors()
    x_sf, v = t["x_sf"].requires_grad_(), torch.zeros(5, 256, dtype=BF, requires_grad=True)
    for call in (lambda: m.Fp8Linear(144, 272, device=CPU).forward(t["x"], x_sf, t["w"], t["w_sf"]), lambda: m.Fp8Quant(256, device=CPU).forward(v),
                 lambda: m.Fp8Quant(256, device=CPU).weights(v)):
        with pytest.warns(UserWarning, match="no part in autograd"):
            with pytest.raises(RuntimeError, match="CPU"):
                call()
        with warnings.catch_warnings(), torch.no_grad():
            warnings.simplefilter("error")
            with pytest.raises(RuntimeError, match="CPU"):
                call()
