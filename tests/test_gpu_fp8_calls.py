"""How the FP8 linear, the quantiser and routing with groups are called: as the first call of a process and in a capture, for a stream of its
own, while another device is current, with an added input that is the output, with more tokens than 32-bit sums of blocks' costs hold."""
import os
import subprocess
import sys

import pytest
import torch

from fp8_ref import BF, DEV, close, product, random_codes, up, values

pytestmark = pytest.mark.gpu
T, N, K = 1531, 2048, 1040


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def calls(m):
    """Name -> (operator, its call on a stream with outputs given or made, the tensor of them that is looked at)"""
    lin, quant, route = m.Fp8Linear(K, N, device=DEV), m.Fp8Quant(N, device=DEV), m.Router(256, 8, groups=8, topk_groups=4, logits_dtype=BF, device=DEV)
    glu = m.Fp8Quant(N // 2, act="swiglu", device=DEV)
    x, x_sf = random_codes(T, K, 1, 128, 1)
    w, w_sf = random_codes(N, K, 128, 128, 2, scale=1 / K)
    dy, dy_sf = random_codes(T, N, 1, 128, 3)
    dc, dc_sf = random_codes(T, N, 128, 1, 4)
    xc, xc_sf = random_codes(T, K, 128, 1, 5)
    g = torch.Generator().manual_seed(6)
    v, d, l = (torch.randn(T, n, generator=g).to(DEV).to(BF) for n in (N, N // 2, 256))
    return {"forward": (lin, lambda s, o=None: lin.forward(x, x_sf, w, w_sf, out=o, stream=s), lambda r: r),
            "input": (lin, lambda s, o=None: lin.backward_input(dy, dy_sf, w, w_sf, out=o, stream=s), lambda r: r),
            "weight": (lin, lambda s, o=None: lin.backward_weight(dc, dc_sf, xc, xc_sf, out=o, stream=s), lambda r: r),
            "quant": (quant, lambda s, o=None: quant.forward(v, cols=True, out=o, stream=s), lambda r: r.col_codes),
            "quant weights": (quant, lambda s, o=None: quant.weights(v, out=o, stream=s), lambda r: r.codes),
            "quant backward": (glu, lambda s, o=None: glu.backward(d, v, out=o, stream=s), lambda r: r.codes),
            "route": (route, lambda s, o=None: route.forward(l, out=o, stream=s), lambda r: r.topk_idx)}


NAMES = ["forward", "input", "weight", "quant", "quant weights", "quant backward", "route"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_stream(m, name):
    _, call, look = calls(m)[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    here = look(call(None))
    s.wait_stream(torch.cuda.current_stream())
    out = look(call(s))
    torch.cuda.synchronize()
    assert torch.equal(out, here)
    owner = lambda t: next(g["stream"] for g in torch.cuda.memory_snapshot() if 0 <= t.data_ptr() - g["address"] < g["total_size"])  # noqa: E731
    assert owner(out) == s.cuda_stream and owner(here) == torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("name", NAMES)
def test_another_current_device_is_refused(m, monkeypatch, name):
    """(The operator is made to say that it lives on a second GPU; there need not be one.)"""
    from moe_expert_ffn_gb300 import block
    op, call, _ = calls(m)[name]
    out = call(None)
    torch.cuda.synchronize()
    monkeypatch.setattr(block, "_current_stream", lambda index: 0)
    monkeypatch.setattr(op, "_dev", 1)
    with pytest.raises(RuntimeError, match="cuda:1.*cuda:0"):
        call(None, out)


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
sys.path.insert(0, {tests!r})
import moe_expert_ffn_gb300 as m
import test_gpu_fp8_calls as t
for name, (_, call, look) in t.calls(m).items():
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        held = call(s)
    look(held).zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(look(held), look(call(None))), name
print("first calls", "good")
"""


def test_the_first_call_of_a_process_in_a_capture(m):
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=os.path.dirname(tests), tests=tests)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls good" in r.stdout, r.stdout + r.stderr


def test_weights_that_change_between_replays(m):
    """A captured call reads the weights anew, those that it asks for ahead of the kernel before it too."""
    for tokens in (1, 40, 600):
        op = m.Fp8Linear(K, 512, device=DEV)
        x, x_sf = random_codes(tokens, K, 1, 128, 1)
        w, w_sf = random_codes(512, K, 128, 128, 2, scale=1 / K)
        w2, w2_sf = random_codes(512, K, 128, 128, 3, scale=1 / K)
        out, s, g = op.buffers(tokens), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        held, held_sf = w.clone(), w_sf.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            op.forward(x, x_sf, held, held_sf, out=out, stream=s)
        for a, a_sf in ((w, w_sf), (w2, w2_sf), (w, w_sf)):
            held.copy_(a)
            held_sf.copy_(a_sf)
            g.replay()
            torch.cuda.synchronize()
            close(out, *product(values(x, x_sf, 1, 128), values(a, a_sf, 128, 128), up(K)))


def test_weight_gradient_of_460_million_tokens(m):
    """Codes past 2^31 elements, blocks whose estimated time is beyond 32 bits.  All but some rows of dy are zero, and sums exact there."""
    tokens, n = 460_000_013, 16
    g = torch.Generator(device=DEV).manual_seed(0)
    rows = torch.tensor([0, 1, 127, 128, 134217727, 134217728, 268435455, 268435456, 459999999, tokens - 1], device=DEV)
    dy = torch.zeros(tokens, n, dtype=torch.uint8, device=DEV)
    dy[rows] = torch.randint(0, 120, (len(rows), n), generator=g, device=DEV, dtype=torch.uint8)
    x = torch.randint(0, 120, (tokens, n), generator=g, device=DEV, dtype=torch.uint8)
    dy_sf, x_sf = (torch.rand(up(tokens), n, generator=g, device=DEV) + 0.5 for _ in range(2))
    dw = m.Fp8Linear(n, n, device=DEV).backward_weight(dy, dy_sf, x, x_sf)
    of = lambda q, sf: q[rows].view(torch.float8_e4m3fn).double() * sf[rows // 128].double()  # noqa: E731
    close(dw, *product(of(dy, dy_sf).t(), of(x, x_sf).t(), len(rows)))


@pytest.mark.parametrize("tokens", [5, 40, 700])
def test_an_added_input_that_is_the_output(m, tokens):
    op = m.Fp8Linear(K, 512, device=DEV)
    x, x_sf = random_codes(tokens, K, 1, 128, 1)
    w, w_sf = random_codes(512, K, 128, 128, 2, scale=1 / K)
    buf = torch.randn(2 * tokens, 1024, device=DEV).to(BF)
    first = op.forward(x, x_sf, w, w_sf, add=buf[:tokens, :512].clone())
    both = buf[:tokens, :512]
    op.forward(x, x_sf, w, w_sf, add=both, out=both)
    assert torch.equal(both, first)
    with pytest.raises(m.MoEError):
        op.forward(x, x_sf, w, w_sf, add=buf.view(4 * tokens, 512)[:tokens], out=both)      # the same start, other rows
