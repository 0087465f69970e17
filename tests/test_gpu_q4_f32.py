"""f32 activations of the 4-bit products count with all their 24 bits: the
error in norm, in every form, group and gating."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemv_expert_id_amd as mm
from q4_f32_cases import BOUND, CASES, FORMS, activations, exact, rel, weights

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("form,group,k,gated", CASES)
def test_q4_f32_norm(form, group, k, gated):
    m, n, variant = FORMS[form][0], FORMS[form][1 + gated], FORMS[form][3 + gated]
    w, x = weights(n * (1 + gated), k, group, k), activations(m, k)
    dev, xd, y = [t.to(DEV) for t in w], x.to(DEV), torch.empty(m, n, device=DEV)
    rec = mm.mm_q4_gemv(mm.q4_params(0, 1, m, n, k, group, gated=gated), *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(y),
                        stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert rec.variant == variant
    err = rel(y.cpu(), exact(*(t[0] for t in w), group, x, gated, n))
    print(f"{err:.2e}")
    assert err <= BOUND[gated]


@pytest.mark.parametrize("group,k", [(32, 2080), (64, 1408), (128, 2176)])
@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("counts,n", [([3, 0, 1, 4], 100), ([9, 20, 0, 11], 100), ([200, 17, 190, 73], 2100)])
def test_q4_f32_norm_of_routed_rows(group, k, gated, counts, n):
    """The same rows by expert id and in expert order."""
    E, R = len(counts), sum(counts)
    w, x = weights(n * (1 + gated), k, group, k, E), activations(R, k)
    of = np.repeat(np.arange(E), counts)
    dev, xd = [t.to(DEV) for t in w], x.to(DEV)
    ids = torch.from_numpy(of.astype(np.int32)).to(DEV)
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device=DEV)
    p = mm.q4_params(0, 1, R, n, k, group, n_experts=E, gated=gated)
    y, z = torch.empty(R, n, device=DEV), torch.empty(R, n, device=DEV)
    mm.mm_q4_id_sorted(p, *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(off), mm.buf(y), stream=torch.cuda.current_stream())
    mm.mm_q4_id_direct(p, *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(ids), mm.buf(z), stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = torch.cat([exact(*(t[e] for t in w), group, x[of == e], gated, n) for e in range(E)])
    print(f"{rel(y.cpu(), want):.2e} {rel(z.cpu(), want):.2e}")
    assert rel(y.cpu(), want) <= BOUND[gated] and rel(z.cpu(), want) <= BOUND[gated]
