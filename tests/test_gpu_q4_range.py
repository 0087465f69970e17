"""4-bit products at the ends of the range that include/mm.h allows, in every
form: activations of one sign just below 2^120."""
from __future__ import annotations

import pytest
import torch

import gemv_expert_id_amd as mm
import moe_ref as ref
from test_gpu_moe import Padded, TORCH, gen, q4_case, q4_check, q4_dev, stream

pytestmark = pytest.mark.gpu

# Rows, outputs of each gating and the tile of 4 or 16 tokens and outputs of a
# block that they lead to: k split for few tokens, for many, with two tiles a
# wave (16 bits, not gated), and the form whose waves share x.
FORMS = {"narrow": (3, 40, 40), "split": (13, 40, 40), "split2": (61, 4100, 0), "block": (61, 16290, 8150)}


def variant(form, gated):
    return {"narrow": 4 + 256 * 16, "split": 16 + 256 * 16, "split2": 16 + 256 * 32,
            "block": 16 + 256 * (64 if gated else 128)}[form]


def run_q4(dt, sdt, case, group, x, n, gated, form):
    m, k = x.shape
    dev, xd, y = q4_dev(case), x.to("cuda:0"), Padded(m, n, TORCH[dt])
    rec = mm.mm_q4_gemv(mm.q4_params(dt, sdt, m, n, k, group, gated=gated), *(mm.buf(t) for t in dev), mm.buf(xd), y.buf,
                        stream=stream())
    assert rec.variant == variant(form, gated)
    out = y.cpu()
    y.untouched()
    return out


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt,gated,form", [(dt, gated, form) for dt in (0, 2) for gated in (0, 1) for form in FORMS
                                           if form != "split2" or (dt and not gated)])
def test_q4_of_large_activations(dt, gated, form, group):
    m, n = FORMS[form][0], FORMS[form][1 + gated]
    k = 3 * group
    codes, scales, biases = q4_case(1, n * (1 + gated), k, group, 2, group)
    if gated:  # gates about 2^64 and ups about 2^58: their product is finite
        for t in (scales, biases):
            t[:, :n] *= 2.0 ** -60
            t[:, n:] *= 2.0 ** -66
    # one sign a row, magnitudes in [2^119, 2^120)
    x = (1 + torch.rand(m, k, generator=gen(k)) * 0.99) * 2.0 ** 119
    x[1::2] *= -1
    x = x.to(TORCH[dt])
    assert float(x.abs().max()) < 2.0 ** 120
    want, err = ref.q4_product(codes[0], scales[0], biases[0], group, x, bool(gated), dt == 0)
    assert float(want.abs().max()) < torch.finfo(TORCH[dt]).max
    got = run_q4(dt, 2, (codes, scales, biases), group, x, n, gated, form)
    q4_check(got, dt, want, err, "y")


@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt,gated,form", [(dt, gated, form) for dt in (0, 1, 2) for gated in (0, 1) for form in FORMS
                                           if form != "split2" or (dt and not gated)])
def test_q4_of_rows_that_are_not_finite(dt, gated, form, group, bad):
    """One activation that is not finite makes its row's outputs NaN and no other's; its place in the row does not matter."""
    m, n = FORMS[form][0], FORMS[form][1 + gated]
    k = 9 * group
    case = q4_case(1, n * (1 + gated), k, group, 1, group)
    case[1][:, ::7] = 0.0  # also where a scale is 0
    x = torch.randn(m, k, generator=gen(k)).to(TORCH[dt])
    clean = run_q4(dt, 1, case, group, x, n, gated, form)
    assert bool(torch.isfinite(clean).all())
    for row, at in ((1, 0), (m - 1, k - 1), (0, k // 2 + 1)):
        z = x.clone()
        z[row, at] = float(bad)
        got = run_q4(dt, 1, case, group, z, n, gated, form)
        assert bool(torch.isnan(got[row]).all())
        keep = [i for i in range(m) if i != row]
        assert torch.equal(got[keep], clean[keep])
