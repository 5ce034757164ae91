"""References in 64 bits for the FP8 linear and quantiser, shared by their tests.

E4M3 codes and f32 scales are exact numbers; a product of two codes is exact in f32.  The kernels sum 128 of them in f32 (at most
128 steps, each within 2^-23 of the running magnitude: 2^-16 of the sum of magnitudes), multiply by the two scales (2^-23 together)
and add up the blocks in f32 (2^-24 of the running magnitude a step): so sums are within (2^-16 + 2^-22 + blocks 2^-24) of the sum
of magnitudes.  One product more or less of K is 1/K of it, K below 2^13 in these tests.
"""
import math

import torch

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def up(n):
    return (n + 127) // 128


def values(codes, sf, br, bc):
    """The numbers that codes [R, C] under scales of br x bc stand for."""
    R, C = codes.shape
    r, c = torch.arange(R, device=codes.device) // br, torch.arange(C, device=codes.device) // bc
    return codes.view(torch.float8_e4m3fn).double() * sf.double()[r][:, c]


def random_codes(R, C, br, bc, seed, scale=1.0):
    """Random codes of every size but NaN, some of them zero, and scales that differ by some powers of two."""
    g = torch.Generator().manual_seed(seed)
    q = (2.0 * torch.randn(R, C, generator=g)).to(torch.float8_e4m3fn).view(torch.uint8)
    wild = torch.randint(0, 256, (R, C), generator=g).to(torch.uint8)
    wild[(wild & 127) == 127] = 0
    q = torch.where(torch.rand(R, C, generator=g) < 0.05, wild, q)
    sf = scale * torch.exp2(2.0 * torch.randn(-(-R // br), -(-C // bc), generator=g)) * (1 + torch.rand(-(-R // br), -(-C // bc), generator=g))
    return q.to(DEV), sf.to(DEV)


def product(a, b, blocks):
    """a [R, D] b [C, D]^T and the bound on the error of its f32 sums."""
    return a @ b.t(), (2.0 ** -16 + 2.0 ** -22 + blocks * 2.0 ** -24) * (a.abs() @ b.abs().t())


def swiglu(y, err, clamp=math.inf):
    """silu(gate) up of [T, 2n]: silu's slope is at most 1.1, its own f32 error 2^-20 of it (exponential, quotient; 2^-149
    of the sigmoid where that is no normal number), the product's rounding 2^-24."""
    n = y.shape[1] // 2
    g, u, eg, eu = y[:, :n].clamp(-clamp, clamp), y[:, n:].clamp(-clamp, clamp), err[:, :n], err[:, n:]
    s = g * torch.sigmoid(g)
    out = s * u
    return out, 1.1 * eg * u.abs() + s.abs() * eu + 1.1 * eg * eu + 2.0 ** -19 * out.abs() + 2.0 ** -148 * (g * u).abs()


def close(got, y, err, what=""):
    u = 2.0 ** -8 if got.dtype == BF else 2.0 ** -23
    assert got.shape == y.shape
    tol = u * y.abs() + err * (1 + u) + 1e-38
    off = (got.double() - y).abs()
    assert (off <= tol).all(), f"{what}: {int((off > tol).sum())} of {y.numel()} off, worst {(off / tol).max().item():.3g} x tolerance"


def close_codes(codes, sf, v, err, br, bc, what=""):
    """Codes and scales of values v known within err: scales are the largest magnitude / 448, codes the nearest E4M3 numbers."""
    R, C = v.shape
    pad = (0, -C % bc, 0, -R % br)
    blocks = lambda t: torch.nn.functional.pad(t, pad).reshape(up_to(R, br), br, up_to(C, bc), bc)  # noqa: E731
    amax, worst = blocks(v.abs()).amax((1, 3)), blocks(err).amax((1, 3))
    assert sf.shape == amax.shape
    assert ((sf.double() - amax / 448).abs() <= worst / 448 + 2.0 ** -23 * amax / 448 + 2.0 ** -149).all(), what
    each = sf.double()[torch.arange(R, device=v.device) // br][:, torch.arange(C, device=v.device) // bc]
    # half a step: 2^-4 of the value where it is normal, 2^-10 of the scale below; the quotient is within 2^-22 of itself; a scale
    # below the normal numbers is rounded by up to 2^-150, and a code, at most 448, multiplies that (or saturates by as much)
    tol = (2.0 ** -4 * v.abs()).maximum(2.0 ** -10 * each) * (1 + 2.0 ** -20) + 2 * err + 2.0 ** -21 * v.abs() + 448 * 2.0 ** -149
    off = (codes.view(torch.float8_e4m3fn).double() * each - v).abs()
    assert (off <= tol).all(), f"{what}: worst {(off / tol).max().item():.3g} x tolerance"


def up_to(n, m):
    return (n + m - 1) // m
