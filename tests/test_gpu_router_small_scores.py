"""Grouped routing by sigmoid scores below the normal f32 numbers (logits under -87.3): the score is rounded once, so keys that tie do,
and a score is the f32 next to the exact sigmoid.

The reference's sigmoid in 64 bits is within 2^-52 of itself; converted to f32 it is the next f32 unless it lies that close to the
middle of two, which the fixed seeds here do not meet (every value's distance is checked)."""
import pytest
import torch

from test_gpu_router_groups import DEV, F32, m, ref_choice  # noqa: F401

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -149


def units(l):
    """Exact sigmoids in units of the smallest f32, none of them within 2^-20 of a unit of the middle of two."""
    s = torch.sigmoid(l.double()) / UNIT
    assert ((s - s.floor() - 0.5).abs() > 2.0 ** -20).all()
    return s.round()


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("lo,hi", [(-88.5, -87.4), (-92.0, -88.0), (-100.0, -90.0)])
def test_ties_made_by_a_bias(m, seed, lo, hi):  # noqa: F811
    """Neighbouring experts 2 j and 2 j + 1 have the same key, a small number of units; keys of different j differ by some units.
    All sums are exact, so a score that is off by one unit changes the order."""
    E, groups, k = 1024, 32, 32
    g = torch.Generator().manual_seed(seed)
    l = (lo + (hi - lo) * torch.rand(1, E, generator=g, dtype=torch.float64)).float()
    s = units(l)[0]
    key = (1 << 20) + torch.randperm(E // 2, generator=g).double().repeat_interleave(2)
    bias = ((key - s) * UNIT).float()
    assert torch.equal(bias.double() / UNIT, key - s)
    l, bias = l.to(DEV), bias.to(DEV)
    for use in (31, 16):
        r = m.Router(E, k, score="sigmoid", bias_on="score", groups=groups, topk_groups=use, device=DEV)
        got = r.forward(l, bias).topk_idx
        assert torch.equal(got, ref_choice(l, bias, k, groups, use, "max", True))
        if use == 31:   # best pairs of the groups that are left, in order
            pairs = got[0].view(-1, 2)
            assert torch.equal(pairs[:, 0] + 1, pairs[:, 1]) and (pairs[:, 0] % 2 == 0).all()


@pytest.mark.parametrize("kind", ["max", "top2"])
@pytest.mark.parametrize("groups,size", [(8, 32), (8, 8), (16, 16)])
def test_random_logits(m, groups, size, kind):  # noqa: F811
    """No bias: from normal scores over those of a few units to zeros, which all tie."""
    T, E = 1500, groups * size
    g = torch.Generator().manual_seed(size)
    l = -86.0 - 20.0 * torch.rand(T, E, generator=g)
    units(l)
    l = l.to(DEV)
    for k in (1, 8):
        r = m.Router(E, k, score="sigmoid", bias_on="score", groups=groups, topk_groups=groups // 2, group_score=kind, device=DEV)
        assert torch.equal(r.forward(l).topk_idx, ref_choice(l, None, k, groups, groups // 2, kind, True))
