"""Router's groups as the constructor takes them: what the library refuses is refused with words of its own where Python checks first."""
import pytest
import torch

CPU = torch.device("cpu")


@pytest.fixture(scope="module")
def m():
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


@pytest.mark.parametrize("groups", [1, 0, -1])
def test_one_group_is_no_limit(m, groups):
    with pytest.raises(ValueError, match="2 or more.*leave both out"):
        m.Router(64, 4, groups=groups, topk_groups=1, device=CPU)


def test_all_groups(m):
    assert m.Router(64, 4, groups=2, topk_groups=2, device=CPU).cfg.topk_groups == 2
