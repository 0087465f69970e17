"""The norm bound of the f32 4-bit products tells activations of fewer bits
from whole ones, at every case that the GPU test runs."""
from __future__ import annotations

import pytest
import torch

from q4_f32_cases import BOUND, CASES, FORMS, activations, exact, rel, weights


def upper(x, bits):
    """x with its lowest `bits` bits cut off."""
    return (x.view(torch.int32) & -(1 << bits)).view(torch.float32)


def parts(x, n):
    """The first n of the bf16 parts that an f32 splits into."""
    out, rest = torch.zeros_like(x), x
    for _ in range(n):
        p = upper(rest, 16)
        out, rest = out + p, rest - p
    return out


@pytest.mark.parametrize("form,group,k,gated", CASES)
def test_norm_bound_tells_missing_bits(form, group, k, gated):
    m, n = FORMS[form][0], 96  # a part of the outputs
    c, s, b = (t[0] for t in weights(n * (1 + gated), k, group, k))
    x = activations(m, k)
    assert torch.equal(parts(x, 3), x)
    want = exact(c, s, b, group, x, gated, n)
    for fewer in (parts(x, 2), parts(x, 1), x.half().float(), x.bfloat16().float()):
        assert rel(exact(c, s, b, group, fewer, gated, n), want) > 2 * BOUND[gated]
