"""The FP8 operators at the ends of what they accept: 16 and 2^20 features, one row, sixteen columns, calls of two threads at once."""
import threading

import pytest
import torch

from fp8_ref import BF, DEV, F32, close, close_codes, product, random_codes, swiglu, up, values

pytestmark = pytest.mark.gpu
MOST = 1 << 20


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    yield mod
    assert mod.lib().moe_fp8_linear_status() == mod.MOE_OK


def codes(R, C, br, bc, seed, scale=1.0):
    """random_codes, made on the device (none of them NaN)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = (2.0 * torch.randn(R, C, generator=g, device=DEV)).to(torch.float8_e4m3fn).view(torch.uint8)
    return q, scale * (0.5 + torch.rand(-(-R // br), -(-C // bc), generator=g, device=DEV))


@pytest.mark.parametrize("T", [1, 20, 130, 300])
@pytest.mark.parametrize("N,K", [(MOST, 16), (16, MOST), (16, 16)])
def test_forward_and_gradients(m, T, N, K):
    x, x_sf = codes(T, K, 1, 128, 1)
    w, w_sf = codes(N, K, 128, 128, 2, scale=1 / K)
    X, W = values(x, x_sf, 1, 128), values(w, w_sf, 128, 128)
    op = m.Fp8Linear(K, N, out_dtype=F32, device=DEV)
    close(op.forward(x, x_sf, w, w_sf), *product(X, W, up(K)))
    dy, dy_sf = codes(T, N, 1, 128, 3)
    close(op.backward_input(dy, dy_sf, w, w_sf), *product(values(dy, dy_sf, 1, 128), W.t(), up(N)))
    dc, dc_sf = codes(T, N, 128, 1, 4)
    xc, xc_sf = codes(T, K, 128, 1, 5)
    close(op.backward_weight(dc, dc_sf, xc, xc_sf), *product(values(dc, dc_sf, 128, 1).t(), values(xc, xc_sf, 128, 1).t(), up(T)))


@pytest.mark.parametrize("T", [1, 17, 260])
def test_swiglu_of_most_features(m, T):
    K = 144
    x, x_sf = codes(T, K, 1, 128, 1)
    w, w_sf = codes(MOST, K, 128, 128, 2, scale=1 / K)
    y, err = swiglu(*product(values(x, x_sf, 1, 128), values(w, w_sf, 128, 128), up(K)))
    o = m.Fp8Linear(K, MOST, act="swiglu", quant="fp8", device=DEV).forward(x, x_sf, w, w_sf)
    close_codes(o.codes, o.sf, y, err, 1, 128)


@pytest.mark.parametrize("T", [1, 129])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_quantiser(m, T, dt):
    v = torch.randn(T, MOST, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(dt)
    none = torch.zeros(T, MOST, dtype=torch.float64, device=DEV)
    o = m.Fp8Quant(MOST, dtype=dt, device=DEV).forward(v, cols=True)
    close_codes(o.codes, o.sf, v.double(), none, 1, 128)
    close_codes(o.col_codes, o.col_sf, v.double(), none, 128, 1)
    w = m.Fp8Quant(MOST, dtype=dt, device=DEV).weights(v)
    close_codes(w.codes, w.sf, v.double(), none, 128, 128)
    few = m.Fp8Quant(16, dtype=dt, device=DEV).forward(v[:, :16], cols=True)
    close_codes(few.codes, few.sf, v[:, :16].double(), none[:, :16], 1, 128)
    close_codes(few.col_codes, few.col_sf, v[:, :16].double(), none[:, :16], 128, 1)


def test_swiglu_quantiser_of_most_columns(m):
    """The two halves of a row are 2^20 columns apart; codes against the same operator on a part of the columns, bit for bit."""
    T, part = 5, 256
    g = torch.Generator(device=DEV).manual_seed(2)
    v, d = torch.randn(T, 2 * MOST, generator=g, device=DEV).to(BF), torch.randn(T, MOST, generator=g, device=DEV).to(BF)
    whole, few = (m.Fp8Quant(n, act="swiglu", device=DEV) for n in (MOST, part))
    o, b = whole.forward(v, cols=True), whole.backward(d, v)
    for at in (0, MOST - part):
        cut = torch.cat([v[:, at:at + part], v[:, MOST + at:MOST + at + part]], 1)
        p, q = few.forward(cut, cols=True), few.backward(d[:, at:at + part], cut)
        assert torch.equal(o.codes[:, at:at + part], p.codes) and torch.equal(o.col_sf[:, at:at + part], p.col_sf)
        for half in (0, 1):
            assert torch.equal(b.codes[:, half * MOST + at:half * MOST + at + part], q.codes[:, half * part:(half + 1) * part])
            assert torch.equal(b.col_codes[:, half * MOST + at:half * MOST + at + part], q.col_codes[:, half * part:(half + 1) * part])


def test_two_threads_at_once(m):
    """Calls of one operator on streams of their own, from two threads."""
    N, K = 2048, 1040
    op = m.Fp8Linear(K, N, device=DEV)
    w, w_sf = random_codes(N, K, 128, 128, 1, scale=1 / K)
    batches = [random_codes(T, K, 1, 128, T) for T in (3, 50, 200, 3000)]
    alone = [op.forward(*b, w, w_sf) for b in batches]
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        for i in range(40):
            out = op.forward(*batches[i % 4], w, w_sf, stream=s)
            s.synchronize()
            if not torch.equal(out, alone[i % 4]):
                wrong.append(i)
        torch.cuda.synchronize()

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not any(t.is_alive() for t in threads) and not wrong


@pytest.mark.parametrize("E,groups,use,k", [(1024, 32, 31, 32), (1024, 2, 1, 32), (32, 32, 5, 5), (4, 2, 1, 2), (992, 31, 2, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_routing_of_most_experts(m, E, groups, use, k, score):
    """Distinct logits far apart: the choice by a stable sort, a group's rank by its largest."""
    T = 70
    g = torch.Generator().manual_seed(E + groups)
    l = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float().div(E / 8).sub(4).to(DEV)
    r = m.Router(E, k, score=score, groups=groups, topk_groups=use, device=DEV).forward(l)
    best = torch.sort(l.view(T, groups, -1).amax(2), dim=1, descending=True, stable=True).indices[:, :use]
    on = torch.zeros(T, groups, dtype=torch.bool, device=DEV).scatter_(1, best, True).repeat_interleave(E // groups, 1)
    want = torch.sort(l.masked_fill(~on, float("-inf")), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.topk_idx.long(), want)
