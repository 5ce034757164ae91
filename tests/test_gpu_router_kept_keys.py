"""Router choices where more of the best keys fall to one lane than it keeps in
order: the last of them and the next, which it does not keep, share all bits
but those that the expert's number displaces, and the larger one has the
higher number.  Choices are compared exactly with a stable sort of the keys."""
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


def reference(key, k):
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k].int()


def crowded(T, E, k, seed):
    """Every token: a lane with 3 clear winners and, at the edge of the chosen, two keys a few units in the last place
    apart, the larger at the higher expert; the other k - 4 winners in other lanes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.empty(T, E)
    for t in range(T):
        c = int(torch.randint(0, 32, (1,), generator=g))
        mine = torch.arange(c, E, 32)
        mine = mine[torch.randperm(len(mine), generator=g)[:5]]
        lo, hi = int(mine[3:].min()), int(mine[3:].max())
        base = float(torch.randint(-3, 6, (1,), generator=g)) + 0.5     # low bits zero: a few units keep the high ones
        x[t] = base - 0.5 - torch.rand(E, generator=g)
        lanes = torch.tensor([i for i in range(32) if i != c])[torch.randperm(31, generator=g)[: k - 4]]
        others = lanes + 32 * torch.randint(0, E // 32, (k - 4,), generator=g)
        top = base + 1.0 + torch.randperm(k - 1, generator=g).float()
        x[t, others], x[t, mine[:3]] = top[: k - 4], top[k - 4:]
        a = torch.tensor(base)
        b = (a.view(torch.int32) + int(torch.randint(1, 4, (1,), generator=g))).view(torch.float32)
        x[t, lo], x[t, hi] = torch.minimum(a, b), torch.maximum(a, b)
    return x


@pytest.mark.parametrize("E", [160, 256, 500, 512, 1000, 1024])
@pytest.mark.parametrize("k", [4, 5, 8, 12])
def test_edge_in_a_crowded_lane(m, E, k):
    T = 96
    x = crowded(T, E, k, seed=E + k).to(DEV)
    ref = reference(x, k)
    assert torch.equal(m.Router(E, k, device=DEV).forward(x).topk_idx, ref)
    bias = torch.zeros(E, device=DEV)
    assert torch.equal(m.Router(E, k, score="sigmoid", device=DEV).forward(x, bias).topk_idx, ref)
    out = m.Router(E, k, balance_coef=1.0, max_tokens=T, device=DEV).forward_train(x)
    assert torch.equal(out.topk_idx, ref)
    assert np.array_equal(out.counts.cpu().numpy()[0], np.bincount(ref.cpu().numpy().reshape(-1), minlength=E))


@pytest.mark.parametrize("value", [1.0, -1.0])
def test_four_kept_and_a_fifth(m, value):
    """The smallest such row, written out: experts 0, 32, 64, 96 and 128 are one lane's."""
    x = torch.full((1, 256), -5.0)
    x[0, [0, 32, 64]] = torch.tensor([10.0, 9.0, 8.0])
    x[0, 96] = value
    x[0, 128] = torch.nextafter(torch.tensor(value), torch.tensor(2.0))
    out = m.Router(256, 4, device=DEV).forward(x.to(DEV))
    assert out.topk_idx.cpu().tolist() == [[0, 32, 64, 128]]


@pytest.mark.parametrize("E,k,spread", [(256, 8, 1e-3), (256, 12, 1e-3), (1024, 12, 1e-2), (512, 9, 3e-3)])
def test_common_offset_and_a_small_spread(m, E, k, spread):
    """What a router gives early in training: chosen rows like the above turn up by themselves."""
    T = 200000
    x = 5.0 + spread * torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(E + k), device=DEV)
    assert torch.equal(m.Router(E, k, device=DEV).forward(x).topk_idx, reference(x, k))


@pytest.mark.parametrize("E,k,n", [(256, 8, 3), (256, 8, 6), (1000, 12, 5), (512, 4, 0)])
def test_few_open_experts_in_one_lane(m, E, k, n):
    """Fewer open experts than slots, all in one lane; the rest closed."""
    T = 64
    g = torch.Generator().manual_seed(n)
    x = torch.full((T, E), -torch.inf)
    ref = torch.full((T, k), -1, dtype=torch.int32)
    for t in range(T):
        mine = torch.arange(t % 32, E, 32)
        mine = mine[torch.randperm(len(mine), generator=g)[:n]]
        x[t, mine] = torch.randn(len(mine), generator=g)
        ref[t, :n] = mine[torch.argsort(-x[t, mine])].int()
    out = m.Router(E, k, device=DEV).forward(x.to(DEV))
    assert torch.equal(out.topk_idx.cpu(), ref)
    assert (out.topk_weights.cpu()[:, n:] == 0).all()
