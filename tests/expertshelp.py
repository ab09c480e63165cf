"""The experts' operators in 64 bits, and the inputs and bounds their tests use.

Bounds.  A product in fp32 over n terms is off by at most n * 2^-23 * sum |terms|
(one rounding of at most 2^-24 for each product and each sum, the order left
open), and a bf16 output adds half a step, 2^-8 of its value.  With small whole
numbers every product and every sum below 2^24 is exact in fp32, so those tests
ask for the bits of the correctly rounded result.
"""
import math

import torch

DEV = torch.device("cuda:0")
BF = torch.bfloat16
HALF = 2.0**-8  # half a step of bf16


def offsets_of(counts, skip=0):
    """expert_offsets on the device; `skip` rows in front of the first expert."""
    off = torch.zeros(len(counts) + 1, dtype=torch.int64)
    off[0] = skip
    off[1:] = skip + torch.tensor(counts).cumsum(0)
    return off.to(torch.int32).to(DEV)


def spans(counts, skip=0):
    at, got = skip, []
    for e, n in enumerate(counts):
        got.append((e, at, at + n))
        at += n
    return got


def ints(gen, lo, hi, *shape):
    """Whole numbers in [lo, hi] as bf16 (exact below 257)."""
    return torch.randint(lo, hi + 1, shape, generator=gen, device=DEV).to(BF)


def normal(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(BF)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "relu":
        return torch.clamp(z, min=0)
    return z


def slope64(z, act):
    if act == "silu":
        return torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "relu":
        return (z > 0).double()
    return torch.ones_like(z)


def product64(x, w, sp):
    """x[rows] W[e]^T of every expert, rows outside them 0; and the sum of |terms|."""
    out = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e, a, b in sp:
        out[a:b] = x[a:b].double() @ w[e].double().t()
        mag[a:b] = x[a:b].double().abs() @ w[e].double().abs().t()
    return out, mag


def weight64(d, x, sp, E):
    out = torch.zeros((E, d.shape[1], x.shape[1]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e, a, b in sp:
        out[e] = d[a:b].double().t() @ x[a:b].double()
        mag[e] = d[a:b].double().abs().t() @ x[a:b].double().abs()
    return out, mag


def assert_bits(got, want64, what):
    """`got` is the correctly rounded value of `want64`, which fp32 holds exactly."""
    want = want64.float().to(got.dtype)
    same = got == want
    assert bool(same.all()), f"{what}: {int((~same).sum())} of {same.numel()} values differ"


def assert_within(got, want64, tol, what):
    d = (got.double() - want64).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds, worst "
        f"{float((d / tol.clamp_min(1e-300)).max()):.3g} of the bound")
