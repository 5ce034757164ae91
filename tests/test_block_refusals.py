"""Argument checks of the norm, router and FP4 linear calls: every refusal is
made on the host before anything is launched, so it needs no GPU."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


BAD, UNSUP = -1, -2
P = 1 << 20        # stands for an aligned device pointer; never dereferenced by a refused call


def norm_cfg(m, **kw):
    d = dict(hidden=256, stream_dtype=0, param_dtype=1, gate=0, quant=0, eps=1e-6, residual_scale=1.0)
    return m.NormConfig(*{**d, **kw}.values())


@pytest.mark.parametrize("kw", [dict(hidden=0), dict(hidden=16385), dict(stream_dtype=2), dict(param_dtype=-1), dict(gate=3),
                                dict(quant=3), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf), dict(residual_scale=math.inf),
                                dict(residual_scale=math.nan), dict(quant=1, hidden=192), dict(quant=2, hidden=48)])
def test_norm_config(m, kw):
    assert m.lib().moe_norm_workspace_bytes(norm_cfg(m, **kw), 4) == 0
    io = m.NormIO(residual=P, ld_residual=20000, w_pre=P, n=P, ld_n=20000, codes=P, sf=P)
    assert m.lib().moe_norm_forward(norm_cfg(m, **kw), 4, io, None) == BAD
    assert m.lib().moe_norm_backward(norm_cfg(m, **kw), 4, m.NormGradIO(), P, None) == BAD


def test_norm_workspace(m):
    f = m.lib().moe_norm_workspace_bytes
    assert f(norm_cfg(m), -1) == 0 and f(None, 4) == 0
    assert 0 < f(norm_cfg(m), 0) <= f(norm_cfg(m), 1) <= f(norm_cfg(m), 1000) <= f(norm_cfg(m), 10 ** 6)


FULL = dict(residual=P, ld_residual=256, y=P, ld_y=256, w_post=P, w_pre=P, h=P, ld_h=256, n=P, ld_n=256)


@pytest.mark.parametrize("cfg,change", [
    (dict(), dict(residual=None)), (dict(), dict(h=None)), (dict(), dict(n=None)), (dict(), dict(ld_y=255)),
    (dict(), dict(ld_residual=1)), (dict(), dict(ld_h=0)), (dict(), dict(ld_n=-256)), (dict(), dict(y=None)),
    (dict(), dict(y=None, w_post=None)), (dict(), dict(gate=P)), (dict(gate=1), dict()), (dict(quant=1), dict()),
    (dict(quant=2), dict(codes=P)), (dict(), dict(codes=P, sf=P)), (dict(), dict(w_pre=None)),
    (dict(), dict(w_post=None, rstd_post=P)), (dict(), dict(residual=P + 1)), (dict(), dict(w_pre=P + 2)),
    (dict(stream_dtype=1), dict(h=P + 2)), (dict(quant=1), dict(codes=P + 1, sf=P)), (dict(quant=1), dict(codes=P, sf=P + 2)),
    (dict(), dict(rstd_pre=P + 1)), (dict(), dict(y=None, w_post=None, h=None, w_pre=None, n=None))])
def test_norm_forward_refuses(m, cfg, change):
    assert m.lib().moe_norm_forward(norm_cfg(m, **cfg), 4, m.NormIO(**{**FULL, **change}), None) == BAD


def test_norm_null_and_counts(m):
    L = m.lib()
    assert L.moe_norm_forward(None, 4, m.NormIO(**FULL), None) == BAD
    assert L.moe_norm_forward(norm_cfg(m), 4, None, None) == BAD
    assert L.moe_norm_forward(norm_cfg(m), -1, m.NormIO(**FULL), None) == BAD
    assert L.moe_norm_forward(norm_cfg(m), 0, m.NormIO(**FULL), None) == 0


GRAD = dict(h=P, ld_h=256, y=P, ld_y=256, w_post=P, w_pre=P, rstd_post=P, rstd_pre=P, dh=P, ld_dh=256, dn=P, ld_dn=256,
            dresidual=P, ld_dresidual=256, dy=P, ld_dy=256, dw_post=P, dw_pre=P)


@pytest.mark.parametrize("cfg,change", [
    (dict(), dict(h=None)), (dict(), dict(dresidual=None)), (dict(), dict(dy=None)), (dict(), dict(dw_post=None)),
    (dict(), dict(dw_pre=None)), (dict(), dict(rstd_post=None)), (dict(), dict(rstd_pre=None)), (dict(), dict(dn=None)),
    (dict(), dict(w_pre=None, dw_pre=None)), (dict(), dict(dh=None, dn=None, w_pre=None, dw_pre=None, rstd_pre=None)),
    (dict(), dict(y=None)), (dict(gate=1), dict()), (dict(gate=1), dict(gate=P)), (dict(), dict(gate=P, dgate=P)),
    (dict(), dict(dgate=P)), (dict(), dict(ld_dy=100)), (dict(), dict(ld_h=100)), (dict(), dict(dw_pre=P + 1)), (dict(), dict(dn=P + 1))])
def test_norm_backward_refuses(m, cfg, change):
    assert m.lib().moe_norm_backward(norm_cfg(m, **cfg), 4, m.NormGradIO(**{**GRAD, **change}), P, None) == BAD


def test_norm_backward_workspace_refused(m):
    f = m.lib().moe_norm_backward
    assert f(norm_cfg(m), 4, m.NormGradIO(**GRAD), None, None) == BAD
    assert f(norm_cfg(m), 4, m.NormGradIO(**GRAD), P + 128, None) == BAD
    assert f(norm_cfg(m), -4, m.NormGradIO(**GRAD), P, None) == BAD


def router_cfg(m, **kw):
    d = dict(num_experts=64, topk=4, score=0, renormalize=1, logits_dtype=1, weight_scale=1.0, balance_coef=0.0, z_coef=0.0)
    return m.RouterConfig(*{**d, **kw}.values())


@pytest.mark.parametrize("kw", [dict(num_experts=0), dict(num_experts=1025), dict(topk=0), dict(topk=33), dict(topk=65), dict(score=2),
                                dict(logits_dtype=2), dict(weight_scale=math.nan), dict(balance_coef=math.inf), dict(z_coef=math.nan),
                                dict(score=1, z_coef=0.1)])
def test_router_config(m, kw):
    L, c = m.lib(), router_cfg(m, **kw)
    assert L.moe_router_workspace_bytes(c, 10, 1) == 0
    assert L.moe_router_forward(c, 4, P, 2000, None, P, P, None, None, None) == BAD
    assert L.moe_balance_loss(c, 4, P, 2000, P, m.BalanceIO(1, None, P, P, P, P), P, None) == BAD
    assert L.moe_router_backward(c, 4, P, 2000, P, P, None, None, P, 2000, None) == BAD


def test_router_refuses(m):
    L, c = m.lib(), router_cfg(m)
    ws = L.moe_router_workspace_bytes
    assert ws(c, -1, 1) == 0 and ws(c, 1, 0) == 0 and 0 < ws(c, 0, 1) <= ws(c, 10 ** 6, 1) <= ws(c, 10 ** 6, 50)
    f = L.moe_router_forward
    assert f(None, 4, P, 64, None, P, P, None, None, None) == BAD
    for args in ((-1, P, 64, None, P, P), (4, None, 64, None, P, P), (4, P, 63, None, P, P), (4, P, 64, None, None, P),
                 (4, P, 64, None, P, None), (4, P + 2, 64, None, P, P), (4, P, 64, P + 1, P, P), (4, P, 64, None, P + 1, P),
                 (4, P, 64, None, P, P + 2)):
        assert f(c, *args, None, None, None) == BAD, args
    assert f(c, 0, P, 64, None, P, P, None, None, None) == 0
    good = dict(num_seqs=2, seq_offsets=P, loss=P, counts=P, prob_mean=P, seq_tokens=P)
    for change in (dict(num_seqs=0), dict(seq_offsets=None), dict(loss=None), dict(counts=None), dict(prob_mean=None),
                   dict(seq_tokens=None), dict(seq_offsets=P + 1), dict(loss=P + 2), dict(counts=P + 1)):
        io = m.BalanceIO(**{**good, **change})
        assert f(c, 4, P, 64, None, P, P, io, P, None) == BAD, change
        assert L.moe_balance_loss(c, 4, P, 64, P, io, P, None) == BAD, change
    io = m.BalanceIO(**good)
    assert f(c, 4, P, 64, None, P, P, io, None, None) == BAD
    assert f(c, 4, P, 64, None, P, P, io, P + 64, None) == BAD
    assert L.moe_balance_loss(c, 4, P, 64, P, None, P, None) == BAD
    assert L.moe_balance_loss(c, 4, P, 64, None, io, P, None) == BAD
    b = L.moe_router_backward
    for args in ((4, P, 64, P, None, None, None, P, 64), (4, None, 64, P, P, None, None, P, 64), (4, P, 64, None, P, None, None, P, 64),
                 (4, P, 64, P, P, None, P, P, 64), (4, P, 64, P, P, None, None, None, 64), (4, P, 60, P, P, None, None, P, 64),
                 (4, P, 64, P, P, None, None, P, 60), (4, P, 64, P, P + 1, None, None, P, 64), (4, P, 64, P, P, None, None, P + 2, 64),
                 (-2, P, 64, P, P, None, None, P, 64)):
        assert b(c, *args, None) == BAD, args
    assert b(c, 4, P, 64, P, P, m.BalanceIO(**{**good, "counts": None}), P, P, 64, None) == BAD


def linear_cfg(m, **kw):
    d = dict(in_features=64, out_features=10, act=0, out_dtype=0, act_clamp=math.inf)
    return m.Fp4LinearConfig(*{**d, **kw}.values())


@pytest.mark.parametrize("kw", [dict(in_features=0), dict(in_features=48), dict(out_features=0), dict(act=2), dict(act=1, out_features=9),
                                dict(out_dtype=3), dict(act_clamp=0.0), dict(act_clamp=math.nan), dict(in_features=-32)])
def test_linear_config(m, kw):
    L, c = m.lib(), linear_cfg(m, **kw)
    assert L.moe_fp4_linear_weight_bytes(c) == 0
    assert L.moe_fp4_linear_transform_weights(c, P, P, P, None) == BAD
    assert L.moe_fp4_linear_forward(c, 1, P, 64, P, None, 0, P, 64, None) == BAD


def test_linear_refuses(m):
    L, c = m.lib(), linear_cfg(m)
    assert L.moe_fp4_linear_weight_bytes(c) >= 10 * 32 + 10 * 2
    t = L.moe_fp4_linear_transform_weights
    for args in ((None, P, P), (P, None, P), (P, P, None), (P + 1, P, P), (P, P, P + 16)):
        assert t(c, *args, None) == BAD, args
    f = L.moe_fp4_linear_forward
    for args in ((-1, P, 64, P, None, 0, P, 10), (1, None, 64, P, None, 0, P, 10), (1, P, 63, P, None, 0, P, 10),
                 (1, P, 64, None, None, 0, P, 10), (1, P, 64, P, P, 9, P, 10), (1, P, 64, P, None, 0, None, 10),
                 (1, P, 64, P, None, 0, P, 9), (1, P + 1, 64, P, None, 0, P, 10), (1, P, 64, P + 16, None, 0, P, 10),
                 (1, P, 64, P, None, 0, P + 1, 10), (1, P, 64, P, P + 1, 10, P, 10)):
        assert f(c, *args, None) == BAD, args
    assert f(c, 17, P, 64, P, None, 0, P, 10, None) == UNSUP
    assert f(c, 0, P, 64, P, None, 0, P, 10, None) == 0


def test_binding_refuses(m):
    """The binding's own checks: types, shapes, devices, pitches, unknown choices."""
    cpu = torch.device("cpu")
    with pytest.raises(ValueError):
        m.BlockNorm(256, gate="row", device=cpu)
    with pytest.raises(ValueError):
        m.BlockNorm(256, dtype=torch.float16, device=cpu)
    with pytest.raises(m.MoEError):
        m.BlockNorm(200, quant="fp8", device=cpu)
    op = m.BlockNorm(256, device=cpu)
    x, w = torch.zeros(3, 256, dtype=torch.bfloat16), torch.ones(256)
    for bad in (dict(residual=x.float(), w_pre=w), dict(residual=x[:, :255], w_pre=w), dict(residual=x, w_pre=w[:10]),
                dict(residual=x, w_pre=w.to(torch.bfloat16)), dict(residual=x.t().contiguous().t(), w_pre=w),
                dict(residual=x, y=x[:2], w_pre=w), dict(residual=x[:1].expand(3, 256), w_pre=w)):
        with pytest.raises(ValueError):
            op.forward(**bad)
    with pytest.raises(ValueError):
        m.Router(8, 2, score="tanh", device=cpu)
    with pytest.raises(m.MoEError):
        m.Router(8, 9, device=cpu)
    r = m.Router(8, 2, balance_coef=1.0, max_tokens=4, device=cpu)
    for call in (lambda: r.forward(torch.zeros(3, 9)), lambda: r.forward(torch.zeros(3, 8, dtype=torch.bfloat16)),
                 lambda: r.forward_train(torch.zeros(5, 8)), lambda: m.Router(8, 2, device=cpu).forward_train(torch.zeros(1, 8)),
                 lambda: r.forward(torch.zeros(3, 8), bias=torch.zeros(7)),
                 lambda: r.forward_train(torch.zeros(3, 8), None, torch.zeros(3, dtype=torch.int32)),
                 lambda: r.balance_loss(torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(m.MoEError):
        m.Fp4Linear(40, 8, device=cpu)
    lin = m.Fp4Linear(64, 8, device=cpu)
    with pytest.raises(ValueError):
        lin.transform_weights(torch.zeros(8, 32), torch.zeros(8, 2, dtype=torch.uint8))
    with pytest.raises(m.MoEError):
        lin.forward(torch.zeros(1, 64, dtype=torch.bfloat16))
    assert ctypes.sizeof(m.NormIO) == 8 * 15 and ctypes.sizeof(m.BalanceIO) == 8 * 6


def test_binding_checks_outputs(m):
    """Outputs are checked like inputs, at every call: types, shapes, pitches, what is missing, what is no tensor."""
    cpu, bf = torch.device("cpu"), torch.bfloat16
    op = m.BlockNorm(256, gate="token", quant="ue8m0", device=cpu)
    x, w, g = torch.zeros(3, 256, dtype=bf), torch.ones(256), torch.ones(3)

    def call(**change):
        o = op.buffers(3)
        for n, v in change.items():
            setattr(o, n, v)
        op.forward(x, x, w_post=w, gate=g, w_pre=w, out=o)

    for change in (dict(h=None), dict(codes=None), dict(sf=None), dict(h=torch.zeros(3, 256)), dict(h=torch.zeros(2, 256, dtype=bf)),
                   dict(n=torch.zeros(3, 128, dtype=bf)), dict(codes=torch.zeros(3, 256, dtype=bf)), dict(sf=torch.zeros(3, 2)),
                   dict(codes=torch.zeros(256, 3, dtype=torch.uint8).t()), dict(rstd_post=torch.zeros(4)),
                   dict(rstd_pre=torch.zeros(3, 1)), dict(h=torch.zeros(1, 256, dtype=bf).expand(3, 256))):
        with pytest.raises(ValueError):
            call(**change)
    with pytest.raises(RuntimeError):   # all is well, but nothing is launched on CPU tensors
        call()
    for bad in (3, "x", [x]):
        with pytest.raises(TypeError):
            op.forward(bad if isinstance(bad, list) else x, x, w_post=bad, gate=g, w_pre=w, out=op.buffers(3))
    with pytest.raises(ValueError):
        op.forward(x, x, w_post=w, gate=torch.ones(256), w_pre=w, out=op.buffers(3))
    with pytest.raises(ValueError):
        op.backward(x, x, x, y=x, w_post=w, gate=g, w_pre=w, rstd_post=torch.ones(3), rstd_pre=torch.ones(2))
    r = m.Router(8, 2, balance_coef=1.0, max_tokens=4, max_seqs=2, device=cpu)
    l = torch.zeros(3, 8)
    o = r.buffers(3, 1)
    for n, v in (("counts", torch.zeros(1, 8)), ("counts", None), ("loss", torch.zeros(2)), ("tokens", torch.zeros(2, dtype=torch.int32)),
                 ("topk_idx", torch.zeros(3, 2, dtype=torch.int64))):
        keep = getattr(o, n)
        setattr(o, n, v)
        with pytest.raises(ValueError):
            r.forward_train(l, out=o)
        setattr(o, n, keep)
    for off in (torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), torch.zeros(2, 2, dtype=torch.int32),
                torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError):
            r.forward_train(l, None, off, out=r.buffers(3, 2))
    with pytest.raises(ValueError):
        r.backward(l, o, d_loss=torch.ones(2))
    with pytest.raises(ValueError):
        r.backward(l, o, d_weights=torch.ones(3, 2, dtype=bf))
