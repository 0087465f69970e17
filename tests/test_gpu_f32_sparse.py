"""f32 products of the feed-forward block over long contractions of which each sum has six
terms: the bound counts these, not the length, so that a missing or misplaced product of
parts shows (without one of the smallest three of six the worst sum is at 14 to 40 times
the bound; over 2048 dense terms it would be at 0.01).

A product lacks at most 2^-21 = 8 U of itself. Each of T terms is rounded by at most T sums
of nonzero numbers, and once more where a wave adds the small products and where waves are
joined; zeros are added exactly. (T + 16) U sum|x w| covers both."""
from __future__ import annotations

import pytest
import torch

import gemv_expert_id_amd as mm
from ffn_ref import U
from test_gpu_f32_small import PRODUCTS
from test_gpu_ffn import F32_SHAPES, GATES, Rows, randn, stream

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TERMS = 6


def sparse(seed, rows, width):
    """Normal values, at most six in a row, the first and the last element among those of every fourth."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = min(TERMS, width)
    at = torch.rand(rows, width, generator=g, device=DEV)
    at[::4, 0], at[::4, -1] = 2, 2
    keep = torch.zeros(rows, width, dtype=torch.bool, device=DEV).scatter_(1, at.topk(n, 1).indices, True)
    return torch.where(keep, randn(seed + 1, rows, width), torch.zeros(1, device=DEV))


def check(got, x, w, what):
    """got = x w^T, one of them with at most 2 TERMS nonzero values in a row."""
    x, w = x.double().contiguous(), w.double().t().contiguous()
    terms = (x != 0).double() @ (w != 0).double()
    assert float(terms.max()) <= 2 * TERMS
    want, absolute = x @ w, x.abs() @ w.abs()
    e = (terms + 16) * U * absolute
    bad = ~((got.double() - want).abs() <= e)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / e)[bad].max()):.3g} of its bound"


@pytest.mark.parametrize("m,n,k", F32_SHAPES + [(9, 40, 8192), (70, 600, 8000), (256, 600, 8004), (300, 1409, 2052), (1037, 2900, 2048), (129, 700, 4099)])
def test_rows(m, n, k):
    for pad in ((4, 1) if k % 4 == 0 else (1,)):
        for x, w in ((sparse(1, m, k), randn(3, 2 * n, k)), (randn(4, m, k), sparse(5, 2 * n, k))):
            X, W = Rows(m, k, torch.float32, k + pad, value=x), Rows(2 * n, k, torch.float32, k + pad, value=w)
            h, pre = Rows(m, n, torch.float32), Rows(m, 2 * n, torch.float32)
            p = mm.gated_params(0, m, n, k, gate=GATES[m % 2], ldx=X.ld, ldw=W.ld)
            mm.mm_gated(p, X.buf, W.buf, h.buf, pre.buf, stream=stream())
            check(pre.t, x, w, "pre")


@pytest.mark.parametrize("m,n,k", PRODUCTS + [(8, 10688, 49), (32, 2048, 130), (70, 5000, 700), (600, 4096, 500), (2816, 200, 260), (4100, 130, 70)])
def test_products(m, n, k):
    """dx over 2n, by rows of dh (two of dpre each) or columns of w; dw over m, by columns of dh or of x."""
    dense = lambda seed, r, c: randn(seed, r, c)  # noqa: E731
    cases = [("dx", sparse(1, m, n), dense(2, m, k), dense(3, 2 * n, k)), ("dx", dense(4, m, n), dense(5, m, k), sparse(6, k, 2 * n).t()),
             ("dw", sparse(7, n, m).t(), dense(8, m, k), dense(9, 2 * n, k)), ("dw", dense(10, m, n), sparse(11, k, m).t(), dense(12, 2 * n, k))]
    for what, dh, x, w in cases:
        d = Rows(m, 2 * n, torch.float32)
        out = Rows(*((m, k) if what == "dx" else (2 * n, k)), torch.float32, k + m % 3)
        X, W = Rows(m, k, torch.float32, out.ld, value=x), Rows(2 * n, k, torch.float32, out.ld, value=w)
        P, D = Rows(m, 2 * n, torch.float32, value=dense(13, m, 2 * n)), Rows(m, n, torch.float32, value=dh)
        p = mm.gated_params(0, m, n, k, gate=GATES[m % 2], ldx=out.ld, ldw=out.ld)
        mm.mm_gated_grad(p, X.buf, W.buf, P.buf, D.buf, d.buf, out.buf if what == "dx" else None, out.buf if what == "dw" else None,
                         stream=stream())
        if what == "dx":
            check(out.t, d.t, w.t(), what)
        else:
            check(out.t, d.t.t(), x.t(), what)
