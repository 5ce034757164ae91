"""moe_router_backward reads the sequences' offsets, counts and sizes: their
addresses are checked on the host like all others."""
import pytest


@pytest.fixture(scope="module")
def m():
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


BAD = -1
P = 1 << 20        # stands for an aligned device pointer; never dereferenced by a refused call
GOOD = dict(num_seqs=2, seq_offsets=P, loss=P, counts=P, prob_mean=P, seq_tokens=P)


@pytest.mark.parametrize("change", [dict(seq_offsets=P + 2), dict(counts=P + 1), dict(seq_tokens=P + 3), dict(num_seqs=(1 << 20) + 1),
                                    dict(num_seqs=0), dict(num_seqs=-1), dict(seq_offsets=None), dict(counts=None), dict(seq_tokens=None)])
def test_loss_arguments(m, change):
    cfg = m.RouterConfig(64, 4, 0, 1, 1, 1.0, 1.0, 0.0)
    io = m.BalanceIO(**{**GOOD, **change})
    assert m.lib().moe_router_backward(cfg, 4, P, 64, None, None, io, P, P, 64, None) == BAD
