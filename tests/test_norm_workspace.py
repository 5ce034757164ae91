"""The workspace of BlockNorm.backward is the call's or its buffers', never
the operator's: nothing that an earlier call uses is given back by a later
one.  (What the kernels do with it is tested on the GPU.)"""
import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def backward(op, T, out=None):
    x, w, r = torch.zeros(T, 256, dtype=BF), torch.ones(256), torch.ones(T)
    return op.backward(x, x, x, w_pre=w, rstd_pre=r, out=out)


def test_workspace_is_the_buffers(m):
    op = m.BlockNorm(256, device="cpu")
    for T in (0, 1, 100, 5000):
        assert op.grad_buffers(T).workspace.numel() >= m.lib().moe_norm_workspace_bytes(op.cfg, T) > 0
    a, b = op.grad_buffers(10), op.grad_buffers(10)
    assert a.workspace.data_ptr() != b.workspace.data_ptr()


def test_operator_keeps_none(m, monkeypatch):
    op = m.BlockNorm(256, device="cpu")
    used = []
    monkeypatch.setattr(op, "_bwd", lambda *a: used.append([t for t in a if torch.is_tensor(t) and t.dtype == torch.uint8]) or 0)
    buf = op.grad_buffers(100, block=False)
    backward(op, 100, buf)
    backward(op, 100)
    backward(op, 1000)
    by_hand = m.NormGrads()
    by_hand.dresidual, by_hand.dw_pre = buf.dresidual, buf.dw_pre
    by_hand.dy = by_hand.dw_post = by_hand.dgate = None
    backward(op, 100, by_hand)
    assert [len(u) for u in used] == [1, 1, 1, 1]
    assert used[0][0] is buf.workspace and len({u[0].data_ptr() for u in used}) == 4
    assert not any(torch.is_tensor(v) for v in vars(op).values())


@pytest.mark.parametrize("bad", [torch.zeros(16, dtype=torch.uint8), torch.zeros(1 << 20), torch.zeros(1 << 10, 1 << 10, dtype=torch.uint8),
                                 torch.zeros(1 << 21, dtype=torch.uint8)[::2]])
def test_workspace_is_checked(m, bad):
    op = m.BlockNorm(256, device="cpu")
    buf = op.grad_buffers(100, block=False)
    buf.workspace = bad
    with pytest.raises(ValueError, match="workspace"):
        backward(op, 100, buf)
    buf.workspace = None                                 # allocated by the call; then all is well but the device
    with pytest.raises(RuntimeError, match="CPU"):
        backward(op, 100, buf)
