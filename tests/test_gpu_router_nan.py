"""The router's gradient where a logit is NaN: the weights are NaN there, in
both forms, and so are their gradients."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemv_expert_id_amd as mm
import moe_ref as ref
from test_gpu_moe import DTYPES, TORCH, U, f64, gen, ids_buf, near, rounding, stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("E", [5, 70, 300])
@pytest.mark.parametrize("renormalize", [0, 1])
def test_topk_grad_of_nan_logits(dt, E, renormalize):
    k = 3
    l = torch.randn(6, E, generator=gen(E)).to(TORCH[dt])
    l[0, E - 1] = float("nan")  # beside experts that are chosen
    l[0, 1] = float("-inf")
    l[1] = float("nan")         # nothing to choose
    l[2, 0], l[2, 2:] = float("nan"), float("-inf")  # one chosen, two slots without an expert
    l[3, 2:] = float("-inf")    # masks alone make no NaN
    l[4, 0] = -float("nan")
    clean = torch.where(torch.isnan(l), torch.full_like(l, float("-inf")), l)
    ids, _ = ref.topk(f64(clean), k, bool(renormalize))
    g = torch.randn(6, k, generator=gen(6))
    ld, di, dg = l.to("cuda:0"), ids_buf(ids), g.to("cuda:0")
    d = torch.full_like(ld, 77.0)
    w, wi = torch.empty(6, k, device="cuda:0"), torch.empty(6, k, dtype=torch.int32, device="cuda:0")
    p = mm.topk_params(dt, 6, E, k, renormalize=renormalize)
    mm.mm_topk(p, mm.buf(ld), mm.buf(wi), mm.buf(w), stream=stream())
    mm.mm_topk_grad(p, mm.buf(ld), mm.buf(di), mm.buf(dg), mm.buf(d), stream=stream())
    torch.cuda.synchronize()
    got, w = f64(d.cpu()), f64(w.cpu())
    np.testing.assert_array_equal(wi.cpu().numpy().view(np.uint32), ids)
    for t in (0, 2, 4):
        chosen = np.zeros(E, dtype=bool)
        chosen[ids[t][ids[t] < E]] = True
        assert np.isnan(w[t][ids[t] < E]).all()
        nan = chosen if renormalize else (l[t].float() != -np.inf).numpy()
        np.testing.assert_array_equal(np.isnan(got[t]), nan)
        assert (got[t][~nan] == 0).all()
    assert (got[1] == 0).all()
    rows = [3, 5]
    want = ref.topk_grad(f64(l)[rows], ids[rows], f64(g)[rows], bool(renormalize))
    # p to 160 steps, the dot product's 6 levels and g - dot, as in test_topk_grad
    scale = np.abs(f64(g)[rows]).max(1, keepdims=True)
    near(got[rows], want, rounding(dt, want) + 400 * U * np.maximum(np.abs(want), 1e-2 * scale), "dlogits")
