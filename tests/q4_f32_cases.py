"""Cases and bound of the f32 4-bit products' error in norm.

In a group an accumulator's value stays about twice the group's part of the
result (the codes carry a 1, q / 16 is half of that), and joins the other groups
at the root of their number. Roundings of 2^-24 at most, evenly spread, are
0.58 * 2^-24 in the root mean square; the upper parts' products are exact in f32
for 32 at a time, so a group of 128 rounds 16 times at the most (eight elements
each), its sum as often, and up to 256 groups are added one after the other, of
which the root of half the number counts:
    0.58 * 2^-24 * (2 * sqrt(16 + 16) + sqrt(256 / 2)) = 7.8e-7.
The gated form multiplies two such results, |silu'| < 1.1: 2.1 times that, and a
few steps. Activations cut to 16 bits are off by 1e-5 in norm, ten times the
bound."""
from __future__ import annotations

import torch

from moe_ref import TORCH

BOUND = {0: 1e-6, 1: 2.2e-6}
# form: rows and outputs (not gated, gated) that lead to it in f32
FORMS = {"narrow": (3, 100, 100, 4 + 256 * 16, 4 + 256 * 16), "split": (13, 100, 100, 16 + 256 * 16, 16 + 256 * 16),
         "block": (61, 16290, 8150, 16 + 256 * 128, 16 + 256 * 64)}
SIZES = [(32, 2080), (64, 2112), (128, 2176), (128, 128), (32, 8192), (64, 4096)]
CASES = [(form, group, k, gated) for form in FORMS for group, k in SIZES for gated in (0, 1)]


def weights(N, k, group, seed, experts=1):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (experts, N, k // 2), generator=g, dtype=torch.int16).to(torch.uint8)
    scales = (torch.rand(experts, N, k // group, generator=g) * 0.02 + 0.001).to(TORCH[1])
    biases = (torch.randn(experts, N, k // group, generator=g) * 0.08).to(TORCH[1])
    return codes, scales, biases


def activations(m, k):
    return torch.randn(m, k, generator=torch.Generator().manual_seed(m + k))


def exact(codes, scales, biases, group, x, gated, n):
    """f64 products of one expert."""
    q = torch.stack((codes % 16, codes // 16), -1).reshape(codes.shape[0], -1).double()
    w = q * scales.double().repeat_interleave(group, 1) + biases.double().repeat_interleave(group, 1)
    y = x.double() @ w.t()
    return y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:] if gated else y


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())
