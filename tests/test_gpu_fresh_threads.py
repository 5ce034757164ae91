"""Calls that are a thread's first: a worker that has touched no GPU yet has no current context, which the driver wants where the
library describes a matrix for bulk copies.  Outputs are made before, so that nothing else binds one."""
import threading

import pytest
import torch

from fp8_ref import DEV, random_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def in_a_thread(f):
    got = []

    def work():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join(timeout=60)
    assert not t.is_alive()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


@pytest.mark.parametrize("T", [1, 40, 700])
@pytest.mark.parametrize("what", ["forward", "input", "weight"])
def test_fp8_linear(m, T, what):
    N, K = 1024, 1040
    op = m.Fp8Linear(K, N, device=DEV)
    x, w = random_codes(T, K, 1, 128, 1), random_codes(N, K, 128, 128, 2, scale=1 / K)
    dy, dc, xc = random_codes(T, N, 1, 128, 3), random_codes(T, N, 128, 1, 4), random_codes(T, K, 128, 1, 5)
    call = {"forward": lambda o=None: op.forward(*x, *w, out=o), "input": lambda o=None: op.backward_input(*dy, *w, out=o),
            "weight": lambda o=None: op.backward_weight(*dc, *xc, out=o)}[what]
    here, out = call(), call()
    out.zero_()
    torch.cuda.synchronize()
    in_a_thread(lambda: call(out))
    torch.cuda.synchronize()
    assert torch.equal(out, here)
    assert in_a_thread(op.device_status) == m.MOE_OK


@pytest.mark.parametrize("T", [4, 600])
def test_the_layer(m, T):
    """(Few tokens: their rows are fetched by a map made in the call.)"""
    import moe_synth
    wl = moe_synth.custom(T, 256, 128, 8, 2)
    i = moe_synth.make_inputs(wl, device="cpu")
    x, x_sf, idx, tw = (i[n].to(DEV) for n in ("x", "x_sf", "topk_idx", "topk_weights"))
    layer = m.MoELayer(T, 256, 128, 8, 2, device=DEV)
    layer.transform_weights(*(i[n].to(DEV) for n in ("w1", "w1_sf", "w2", "w2_sf")))
    y = layer.forward(x, x_sf, idx, tw).clone()
    out = torch.zeros_like(y)
    torch.cuda.synchronize()
    in_a_thread(lambda: layer.forward(x, x_sf, idx, tw, y=out))
    torch.cuda.synchronize()
    assert torch.equal(out, y)
    assert layer.device_status() == m.MOE_OK


@pytest.mark.parametrize("what", ["quant", "route", "groups"])
def test_operators_without_maps(m, what):
    T = 300
    v = torch.randn(T, 256, device=DEV)
    if what == "quant":
        op = m.Fp8Quant(256, dtype=torch.float32, device=DEV)
        here, out = op.forward(v, cols=True), op.buffers(T, cols=True)
        look = lambda o: (o.codes, o.sf, o.col_codes, o.col_sf)  # noqa: E731
        call = lambda: op.forward(v, out=out)  # noqa: E731
    else:
        op = m.Router(256, 8, device=DEV, **(dict(groups=8, topk_groups=4) if what == "groups" else {}))
        here, out = op.forward(v), op.buffers(T)
        look = lambda o: (o.topk_idx, o.topk_weights)  # noqa: E731
        call = lambda: op.forward(v, out=out)  # noqa: E731
    torch.cuda.synchronize()
    in_a_thread(call)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(look(out), look(here)))
