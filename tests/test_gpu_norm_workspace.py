"""Backward passes of one BlockNorm that are captured, grow, and run on
several streams: each has its own workspace, so none writes into memory that
another one, or anybody else, has been given."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
H = 1024


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def inputs(m, op, T, seed):
    g = torch.Generator().manual_seed(seed)
    x, dn, dh = (torch.randn(T, H, generator=g).to(BF).to(DEV) for _ in range(3))
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(DEV)
    return dict(h=x, dh=dh, dn=dn, w_pre=w, rstd_pre=op.forward(x, w_pre=w).rstd_pre)


def same(a, b):
    return torch.equal(a.dresidual, b.dresidual) and torch.equal(a.dw_pre, b.dw_pre)


@pytest.mark.parametrize("own_buffers", [False, True])
def test_replay_after_a_larger_batch(m, own_buffers):
    op = m.BlockNorm(H, device=DEV)
    d, big = inputs(m, op, 100, 1), inputs(m, op, 3000, 2)
    want = op.backward(**d)
    buf = op.grad_buffers(100, block=False) if own_buffers else None
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        op.backward(**d, out=buf)
        with torch.cuda.graph(g, stream=s):
            out = op.backward(**d, out=buf)
    torch.cuda.synchronize()
    want_big = op.backward(**big)
    fill = [torch.full((1 << 20,), i, dtype=torch.uint8, device=DEV) for i in range(64)]
    out.dresidual.zero_(), out.dw_pre.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert same(out, want) and same(op.backward(**big), want_big)
    assert all((f == i).all() for i, f in enumerate(fill))


def test_growing_batches_on_a_stream(m):
    """Larger and larger batches in order on one stream, while the current stream allocates and writes."""
    op, s = m.BlockNorm(H, device=DEV), torch.cuda.Stream()
    ds = [inputs(m, op, T, T) for T in (10, 100, 1000, 4000)]
    want = [op.backward(**d) for d in ds]
    torch.cuda.synchronize()
    got, fill = [], []
    for d in ds:
        got.append(op.backward(**d, stream=s))
        fill.append(torch.full((8 << 20,), 7, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, want)) and all((f == 7).all() for f in fill)


def test_two_streams_at_once(m):
    op, streams = m.BlockNorm(H, device=DEV), [torch.cuda.Stream() for _ in range(2)]
    ds = [inputs(m, op, 2000, i) for i in range(2)]
    want = [op.backward(**d) for d in ds]
    bufs = [op.grad_buffers(2000, block=False) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, b, s in zip(ds, bufs, streams):
            op.backward(**d, out=b, stream=s)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(bufs, want))
