"""The operators together, as an MoE block uses them (examples/moe_block.py):
a serving step against its parts in 64 bits, its capture into a CUDA graph,
and the router's training.

Tolerance of the step: the routed experts are compared with the layer's own
output on the same inputs (its accuracy has tests of its own); the shared
expert rounds its intermediate to bf16 (2^-8 of each factor, averaged over
`inter` terms of random sign) and its output once: 2^-7 of the output's rms."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("moe_block_example", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def dense(packed):
    w, sf = (t.cpu() for t in packed)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(w & 15).long()], grid[(w >> 4).long()]], 2).reshape(w.shape[0], -1)
    return v * torch.ldexp(torch.ones(()).double(), sf.double() - 127).repeat_interleave(32, 1)


def stream(T, H, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), (0.2 * torch.randn(T, H, generator=g)).to(torch.bfloat16).cuda())


def test_step_is_its_parts(ex):
    T, H, I, E, k = 5, 512, 256, 16, 3
    b = ex.MoEBlock(T, H, I, E, k)
    h0, y0 = stream(T, H)
    h, out = b.step(h0, y0)
    y = y0.double().cpu()
    z = h0.double().cpu() + b.gate.double().cpu() * y * (y.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * b.w_post.double().cpu()
    n = z * (z.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * b.w_pre.double().cpu()
    assert (h.double().cpu() - z).abs().max() <= 2.0 ** -8 * z.abs().max()
    assert (b.normed.n.double().cpu() - n).abs().max() <= 2.0 ** -8 * n.abs().max()
    top = torch.sort(b.logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(b.routed.topk_idx.long(), top)
    routed = b.experts.forward(b.normed.codes, b.normed.sf, b.routed.topk_idx, b.routed.topk_weights).double().cpu()
    x = b.normed.n.double().cpu()
    gu = x @ dense(b.shared["gate_up"]).t()
    mid = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    ref = routed + mid @ dense(b.shared["down"]).t()
    assert (out.double().cpu() - ref).norm() <= 2.0 ** -7 * ref.norm()
    assert b.experts.device_status() == ex.moe.MOE_OK


def test_step_captured(ex):
    T, H, I, E, k = 16, 256, 128, 8, 2
    b = ex.MoEBlock(T, H, I, E, k, seed=3)
    h0, y0 = stream(T, H, seed=4)
    h, out = (t.clone() for t in b.step(h0, y0))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        b.step(h0, y0)
        with torch.cuda.graph(g, stream=s):
            b.step(h0, y0)
    b.out.zero_()
    b.normed.h.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.normed.h, h) and torch.equal(b.out, out)


def test_router_training_balances(ex):
    T, H, I, E, k = 512, 256, 128, 16, 2
    b = ex.MoEBlock(T, H, I, E, k, seed=5)
    b.w_router[0] += 0.05
    g = torch.Generator().manual_seed(6)
    h = (torch.randn(T, H, generator=g) + 1.0).to(torch.bfloat16).cuda()
    y = torch.zeros_like(h)
    first, top0 = b.train_router(h, y, lr=2.0)
    for _ in range(80):
        last, top1 = b.train_router(h, y, lr=2.0)
    assert last[0].item() < 0.9 * first[0].item() and top1 < top0
    assert last[1].item() >= 0.99e-2                     # alpha is the balance loss of a perfectly even batch
