"""The sequences of a training forward belong to its result: a backward pass
that does not repeat them takes the same ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


@pytest.mark.parametrize("offsets", [[5, 40], [0, 11, 50], [0, 50]])
@pytest.mark.parametrize("given", [False, True])
def test_backward_takes_the_forwards_sequences(m, offsets, given):
    T, E, k = 50, 24, 3
    op = m.Router(E, k, balance_coef=2.0, z_coef=0.5, max_tokens=T, max_seqs=2, device=DEV)
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    one = torch.ones((), device=DEV)
    out = op.balance_loss(x, op.forward(x).topk_idx, off) if given else op.forward_train(x, seq_offsets=off)
    d = op.backward(x, out, d_loss=one)
    assert torch.equal(d, op.backward(x, out, d_loss=one, seq_offsets=off))
    outside = torch.ones(T, dtype=torch.bool)
    outside[offsets[0]:offsets[-1]] = False
    assert (d[outside.to(DEV)] == 0).all() and (d[~outside.to(DEV)] != 0).any()


def test_buffers_used_again_without_offsets(m):
    """One set of buffers, a batch with sequences and then one without: each backward pass goes by its own forward."""
    T, E, k = 30, 16, 2
    op = m.Router(E, k, balance_coef=2.0, max_tokens=T, device=DEV)
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(DEV)
    buf, one = op.buffers(T, 1), torch.ones((), device=DEV)
    op.forward_train(x, seq_offsets=torch.tensor([3, 9], dtype=torch.int32, device=DEV), out=buf)
    assert (op.backward(x, buf, d_loss=one)[9:] == 0).all()
    op.forward_train(x, out=buf)
    assert torch.equal(op.backward(x, buf, d_loss=one), op.backward(x, op.forward_train(x), d_loss=one))
    assert (op.backward(x, buf, d_loss=one)[9:] != 0).any()
