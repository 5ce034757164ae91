"""The test hook that makes waits give up arms the calling thread's next FP8 linear call, and no other thread's."""
import threading

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


def test_another_threads_call(m):
    T, N, K = 300, 272, 400
    op = m.Fp8Linear(K, N, device=DEV)
    a = *random_codes(T, K, 1, 128, 1), *random_codes(N, K, 128, 128, 2)
    before = op.forward(*a)
    assert op.device_status() == m.MOE_OK
    assert m.lib().moe_fp8_linear_test_arm_timeout(20000) == m.MOE_OK
    seen = []

    def other():
        out = op.forward(*a)
        seen.append((op.device_status(), torch.equal(out, before)))

    t = threading.Thread(target=other)
    t.start()
    t.join(timeout=60)
    assert seen == [(m.MOE_OK, True)]
    op.forward(*a)                       # this thread's is the armed one
    assert op.device_status() == m.MOE_ERR_DEVICE_TIMEOUT
    assert torch.equal(op.forward(*a), before)
    assert op.device_status() == m.MOE_OK
