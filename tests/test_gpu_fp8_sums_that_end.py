"""Waits that run out where a cluster's CTAs send one another their sums: the call ends, the status says so, and calls before, beside and
after it are as always.  (CTA 0 withholds its copies; what the others send to it lands before it leaves.)"""
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


@pytest.mark.parametrize("T", [1, 2, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("act,quant", [(None, None), ("swiglu", "fp8")])
def test_the_call_after(m, T, act, quant):
    N, K = 512, 7168      # few columns, a long axis: eight CTAs to a tile
    op = m.Fp8Linear(K, N, act=act, quant=quant, device=DEV)
    a = *random_codes(T, K, 1, 128, 1), *random_codes(N, K, 128, 128, 2, scale=1 / K)
    flat = lambda o: torch.cat([o.codes.float(), o.sf], 1) if quant else o  # noqa: E731
    before = flat(op.forward(*a))
    assert op.device_status() == m.MOE_OK
    for _ in range(3):
        assert m.lib().moe_fp8_linear_test_arm_timeout(3000) == m.MOE_OK
        op.forward(*a)
        after = [flat(op.forward(*a)) for _ in range(4)]     # launched while it still waits
        assert op.device_status() == m.MOE_ERR_DEVICE_TIMEOUT
        assert all(torch.equal(t, before) for t in after)
    assert op.device_status() == m.MOE_OK
