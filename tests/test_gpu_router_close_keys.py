"""Router choices that only the last bits of the f32 keys decide: many keys
within a few units in the last place of one another, in one lane's experts and
across lanes, among the chosen and at their edge.  Choices are compared
exactly with a stable sort of the keys."""
import numpy as np
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


def reference(x, bias, k):
    key = x.cpu().numpy() if bias is None else (x + bias).cpu().numpy()
    return np.argsort(-key, axis=1, kind="stable")[:, :k].astype(np.int32)


def near(T, E, base, spread, seed, sign=1.0):
    """base plus whole multiples of its unit in the last place"""
    g = torch.Generator().manual_seed(seed)
    b = torch.full((T, E), base).view(torch.int32)
    return sign * (b + torch.randint(0, spread, (T, E), generator=g, dtype=torch.int32)).view(torch.float32)


@pytest.mark.parametrize("E,k", [(8, 3), (64, 12), (100, 8), (256, 8), (256, 13), (512, 12), (1000, 8), (1000, 32)])
@pytest.mark.parametrize("spread", [2, 40, 3000, 200000])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_units_in_the_last_place(m, E, k, spread, sign):
    T = 200
    x = near(T, E, 1.5, spread, seed=E + spread, sign=sign).to(DEV)
    out = m.Router(E, k, device=DEV).forward(x)
    assert np.array_equal(out.topk_idx.cpu().numpy(), reference(x, None, k))


@pytest.mark.parametrize("E,k", [(256, 8), (512, 6)])
def test_pairs_among_the_chosen_and_at_their_edge(m, E, k):
    """Well separated keys except one pair of neighbours in the sorted order, a unit in the last place apart, at every rank
    up to k + 1, with the larger one at the higher index."""
    T = k + 1
    g = torch.Generator().manual_seed(E)
    x = torch.empty(T, E)
    for t in range(T):
        order = torch.randperm(E, generator=g)
        vals = torch.linspace(3.0, -3.0, E)
        a, b = int(order[t]), int(order[t + 1])
        x[t, order] = vals
        top = x[t, a].clone()
        hi, lo = max(a, b), min(a, b)
        x[t, hi] = top
        x[t, lo] = torch.nextafter(top, torch.tensor(-10.0))
    x = x.to(DEV)
    out = m.Router(E, k, device=DEV).forward(x)
    assert np.array_equal(out.topk_idx.cpu().numpy(), reference(x, None, k))
    bias = torch.zeros(E, device=DEV)
    assert np.array_equal(m.Router(E, k, device=DEV).forward(x, bias).topk_idx.cpu().numpy(), reference(x, bias, k))


@pytest.mark.parametrize("E,k,n", [(256, 8, 4), (256, 8, 5), (256, 8, 8), (512, 12, 5), (512, 12, 12), (1000, 12, 9), (1024, 32, 20)])
def test_chosen_experts_congruent_modulo_32(m, E, k, n):
    """n of the largest keys at experts c, c + 32, c + 64, ...: the experts that one lane of a token's 32 holds."""
    T = 64
    g = torch.Generator().manual_seed(n)
    x = torch.randn(T, E, generator=g)
    for t in range(T):
        rows = torch.arange(t % 32, E, 32)[: min(n, (E - t % 32 + 31) // 32)]
        x[t, rows] = 5.0 + torch.rand(len(rows), generator=g)
    x = x.to(DEV)
    out = m.Router(E, k, balance_coef=1.0, max_tokens=T, device=DEV).forward_train(x)
    ref = reference(x, None, k)
    assert np.array_equal(out.topk_idx.cpu().numpy(), ref)
    assert np.array_equal(out.counts.cpu().numpy()[0], np.bincount(ref.reshape(-1), minlength=E))
