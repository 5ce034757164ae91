"""The FP8 operators together, as a shared expert uses them (examples/shared_expert.py, examples/moe_block.py): a serving step and
a training step against the same chain in 64 bits, micro-batches, capture, and the block with a grouped router.

Tolerances.  The chain is followed stage by stage on the codes that the stage before wrote (fp8_ref.py), so a stage's error is its
own: a product's sums and one bf16 rounding, a quantiser's half step.  Against the chain of unquantised numbers each of the
three quantisations of a product's operands is off by at most 2^-4 of a value, 2^-4 / sqrt(3) in the mean square if
spread evenly, at random: a sum of K such products is off by less than 2^-4 of its root mean square per operand; four operands deep
(x, W, mid, W) and through SwiGLU's slope of at most 1.1 a quarter covers it, where a wrong term would be of order one."""
import importlib.util
import os

import pytest
import torch

from fp8_ref import DEV, close, close_codes, product, swiglu, up, values

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def load(name):
    spec = importlib.util.spec_from_file_location(name + "_example", os.path.join(ROOT, "examples", name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    return load("shared_expert")


def batch(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, generator=g).to(BF).to(DEV), torch.randn(T, H, generator=g).to(BF).to(DEV)


@pytest.mark.parametrize("T", [1, 17, 129, 1000])
def test_serving_step(ex, T):
    H, I = 512, 384
    e = ex.random_expert(H, I)
    x, add = batch(T, H, 1)
    q, mid = bufs = e.buffers(T)
    y = e.forward(x, add=add, buffers=bufs)
    close_codes(q.codes, q.sf, x.double(), torch.zeros(T, H, dtype=torch.float64, device=DEV), 1, 128)
    W1, W2 = values(e.q_gate_up.codes, e.q_gate_up.sf, 128, 128), values(e.q_down.codes, e.q_down.sf, 128, 128)
    close_codes(mid.codes, mid.sf, *swiglu(*product(values(q.codes, q.sf, 1, 128), W1, up(H))), 1, 128)
    ref, err = product(values(mid.codes, mid.sf, 1, 128), W2, up(I))
    ref, err = ref + add.double(), err + 2.0 ** -23 * (ref.abs() + add.double().abs())
    close(y, ref, err)
    v = x.double() @ e.w_gate_up.double().t()
    whole = (torch.nn.functional.silu(v[:, :I]) * v[:, I:]) @ e.w_down.double().t() + add.double()
    assert (y.double() - whole).norm() <= 0.25 * whole.norm()
    out = add.clone()
    assert torch.equal(e.forward(x, add=out, out=out, buffers=bufs), y)


@pytest.mark.parametrize("T", [3, 200, 1025])
def test_training_step(ex, T):
    H, I = 512, 384
    e = ex.random_expert(H, I, seed=2)
    x, dy = batch(T, H, 3)
    y, saved = e.forward_train(x)
    dx, (dw1, dw2) = e.backward(dy, saved)
    W1, W2 = e.w_gate_up.double().requires_grad_(), e.w_down.double().requires_grad_()
    X = x.double().requires_grad_()
    v = X @ W1.t()
    ref = (torch.nn.functional.silu(v[:, :I]) * v[:, I:]) @ W2.t()
    ref.backward(dy.double())
    for got, want in ((y, ref.detach()), (dx, X.grad), (dw1, W1.grad), (dw2, W2.grad)):
        assert got.shape == want.shape
        assert (got.double() - want).norm() <= 0.25 * want.norm()
    # a second micro-batch is added to the first one's gradients, in place
    x2, dy2 = batch(T, H, 4)
    _, saved2 = e.forward_train(x2)
    _, alone = e.backward(dy2, saved2)
    both = dw1.clone(), dw2.clone()
    e.backward(dy2, saved2, grads=both)
    for b, a, c in zip(both, (dw1, dw2), alone):
        assert (b.double() - a.double() - c.double()).abs().max() <= 2.0 ** -22 * (a.abs() + c.abs()).max()
    before = e.q_down.codes.clone()
    e.update((dw1, dw2), lr=0.1)
    assert not torch.equal(before, e.q_down.codes)


def test_training_step_captured(ex):
    T, H, I = 150, 256, 128
    e = ex.random_expert(H, I, seed=5)
    x, dy = batch(T, H, 6)
    _, saved = e.forward_train(x)
    first = e.backward(dy, saved)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            y, saved = e.forward_train(x)
            dx, (dw1, dw2) = e.backward(dy, saved)
    for t in (dx, dw1, dw2):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, first[0]) and torch.equal(dw1, first[1][0]) and torch.equal(dw2, first[1][1])


def test_block_with_groups_and_the_shared_expert(ex):
    mb = load("moe_block")
    T, H, I, E, k = 200, 512, 256, 16, 3
    b = mb.MoEBlock(T, H, I, E, k, groups=4, topk_groups=2)
    h0, y0 = batch(T, H, 7)
    h, out = b.step(h0, y0)
    L = b.logits
    use = torch.sort(L.view(T, 4, 4).amax(2), dim=1, descending=True, stable=True).indices[:, :2]
    on = torch.zeros(T, 4, dtype=torch.bool, device=DEV).scatter_(1, use, True).repeat_interleave(4, 1)
    top = torch.sort(L.masked_fill(~on, float("-inf")), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(b.routed.topk_idx.long(), top)
    routed = b.experts.forward(b.normed.codes, b.normed.sf, b.routed.topk_idx, b.routed.topk_weights)
    assert torch.equal(b.shared.forward(b.normed.n, add=routed), out)
    assert not torch.equal(out, routed)
    assert b.experts.device_status() == mb.moe.MOE_OK and mb.moe.lib().moe_fp8_linear_status() == mb.moe.MOE_OK
