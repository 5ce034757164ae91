"""Fp8Linear.device_status(): what the class says of waits that gave up, for every one of its calls; once, and nothing of good calls."""
import pytest
import torch

from fp8_ref import DEV, random_codes

pytestmark = pytest.mark.gpu
T, N, K = 300, 272, 400


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_expert_ffn_gb300 import build
    build.build()
    import moe_expert_ffn_gb300 as mod
    return mod


@pytest.mark.parametrize("what", ["forward", "input", "weight"])
def test_a_wait_that_gave_up(m, what):
    op, other = m.Fp8Linear(K, N, device=DEV), m.Fp8Linear(16, 16, device=DEV)
    call = {"forward": lambda: op.forward(*random_codes(T, K, 1, 128, 1), *random_codes(N, K, 128, 128, 2)),
            "input": lambda: op.backward_input(*random_codes(T, N, 1, 128, 3), *random_codes(N, K, 128, 128, 2)),
            "weight": lambda: op.backward_weight(*random_codes(T, N, 128, 1, 4), *random_codes(T, K, 128, 1, 5))}[what]
    before = call()
    assert op.device_status() == m.MOE_OK
    assert m.lib().moe_fp8_linear_test_arm_timeout(20000) == m.MOE_OK
    call()
    assert other.device_status() == m.MOE_ERR_DEVICE_TIMEOUT      # of the device, whichever operator asks
    assert op.device_status() == m.MOE_OK
    assert torch.equal(call(), before)
    assert op.device_status() == m.MOE_OK


def test_an_operator_for_the_cpu(m):
    with pytest.raises(RuntimeError, match="CPU"):
        m.Fp8Linear(K, N, device="cpu").device_status()
