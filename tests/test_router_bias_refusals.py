"""What a router's bias may be added to: refusals, made on the host."""
import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


def test_config(m):
    ws = m.lib().moe_router_workspace_bytes
    cfg = lambda score, on: m.RouterConfig(64, 4, score, 1, 1, 1.0, 0.0, 0.0, on)  # noqa: E731
    assert ws(cfg(1, 0), 4, 1) > 0 and ws(cfg(1, 1), 4, 1) > 0 and ws(cfg(0, 0), 4, 1) > 0
    for score, on in ((0, 1), (1, 2), (1, -1), (0, 2)):
        assert ws(cfg(score, on), 4, 1) == 0


def test_names(m):
    with pytest.raises(ValueError, match="bias_on"):
        m.Router(8, 2, score="sigmoid", bias_on="weight", device=torch.device("cpu"))
    with pytest.raises(m.MoEError):
        m.Router(8, 2, score="softmax", bias_on="score", device=torch.device("cpu"))
    assert m.Router(8, 2, score="sigmoid", bias_on="score", device=torch.device("cpu")).cfg.bias_on == 1
    assert m.Router(8, 2, device=torch.device("cpu")).cfg.bias_on == 0
