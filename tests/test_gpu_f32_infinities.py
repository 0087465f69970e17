"""f32 products of the feed-forward block with infinities and NaN: every form gives what the
sum of the products in f32 gives, an infinity where all infinite terms have one sign, and
sums without such terms keep their bits."""
from __future__ import annotations

import pytest
import torch

import gemv_expert_id_amd as mm
from test_gpu_f32_small import PRODUCTS, bound, near, products
from test_gpu_ffn import F32_SHAPES, GATES, Rows, randn, stream

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")


def expected(x, w):
    """x w^T where that is finite, the infinity or NaN that it holds (else 0), and where it is finite."""
    f = lambda b: b.float()  # noqa: E731
    xi, xj, wi, wj = f(x == INF), f(x == -INF), f(w == INF), f(w == -INF)
    plus = xi @ f(w > 0).t() + xj @ f(w < 0).t() + f(x > 0) @ wi.t() + f(x < 0) @ wj.t()
    minus = xi @ f(w < 0).t() + xj @ f(w > 0).t() + f(x < 0) @ wi.t() + f(x > 0) @ wj.t()
    nan = (xi + xj) @ f(w == 0).t() + f(x == 0) @ (wi + wj).t() + f(x.isnan()) @ torch.ones_like(w).t() + torch.ones_like(x) @ f(w.isnan()).t()
    nan = (nan > 0) | ((plus > 0) & (minus > 0))
    odd = torch.zeros_like(plus).masked_fill(plus > 0, INF).masked_fill(minus > 0, -INF).masked_fill(nan, float("nan"))
    return odd, odd == 0


def same(got, x, w, terms, what):
    odd, finite = expected(x, w)
    assert torch.equal(got.isnan(), odd.isnan()), f"{what}: {int((got.isnan() != odd.isnan()).sum())} NaN differ"
    assert torch.equal(got.nan_to_num(0, 0, 0) != got.nan_to_num(0), odd.nan_to_num(0, 0, 0) != odd.nan_to_num(0)), f"{what}: infinities differ"
    assert torch.equal((got == INF), odd == INF) and torch.equal(got == -INF, odd == -INF), f"{what}: infinities differ"
    zero = lambda t: torch.where(t.isfinite(), t, torch.zeros_like(t))  # noqa: E731
    want, absolute = products(zero(x), zero(w))
    bad = finite & ~((got.double() - want).abs() <= bound(want, absolute, terms))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} finite sums off"


def with_infinities(t, seed):
    """Infinities of either sign, a zero, NaN and a NaN whose upper 16 bits are those of an infinity, in a few rows."""
    t = t.clone()
    rows, width = t.shape
    g = torch.Generator().manual_seed(seed)
    at = torch.randint(0, width, (8,), generator=g).tolist()
    put = lambda r, c, v: t.__setitem__((r, c), v) if r < rows else None  # noqa: E731
    put(0, width - 1, INF)
    put(3, at[0], -INF)
    put(rows - 1, 0, INF)
    put(rows // 2, at[1], INF)
    put(rows // 2, at[2], -INF)
    put(5, at[3], float("nan"))
    if rows > 8:
        t.view(torch.int32)[8, at[4]] = 0x7F800001
    put(11, at[5], 0.0)
    put(12, at[6], 2.0 ** -140)
    return t


def forward(x, w, m, n, k, pad):
    X, W = Rows(m, k, torch.float32, k + pad, value=x), Rows(2 * n, k, torch.float32, k + pad, value=w)
    for d, s in ((X, x), (W, w)):  # (a copy on the device might quiet a NaN)
        d.store.view(torch.int32)[d.shift:].as_strided(s.shape, (d.ld, 1)).copy_(s.view(torch.int32))
    h, pre = Rows(m, n, torch.float32), Rows(m, 2 * n, torch.float32)
    p = mm.gated_params(0, m, n, k, gate=GATES[m % 2], ldx=X.ld, ldw=W.ld)
    mm.mm_gated(p, X.buf, W.buf, h.buf, pre.buf, stream=stream())
    return pre.t


@pytest.mark.parametrize("m,n,k", F32_SHAPES)
def test_rows(m, n, k):
    x, w = randn(1, m, k), randn(2, 2 * n, k)
    for pad in ((4, 1) if k % 4 == 0 else (1,)):
        plain = forward(x, w, m, n, k, pad)
        for a, b in ((with_infinities(x, 1), w), (x, with_infinities(w, 2)), (with_infinities(x, 3), with_infinities(w, 4))):
            pre = forward(a, b, m, n, k, pad)
            same(pre, a, b, k, "pre")
            rows = (a == x).all(1)[:, None] & (b == w).all(1)[None]
            assert torch.equal(pre[rows], plain[rows]), "other rows have changed"


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_products(m, n, k):
    """dx and dw of a dpre that holds infinities through dh, and of x and w that do."""
    pre, x, w = randn(1, m, 2 * n), randn(3, m, k), randn(4, 2 * n, k)
    for dh, x, w in ((with_infinities(randn(2, m, n), 5), x, w), (randn(2, m, n), with_infinities(x, 6), with_infinities(w, 7))):
        dpre, dx, dw = Rows(m, 2 * n, torch.float32), Rows(m, k, torch.float32, k + m % 3), Rows(2 * n, k, torch.float32, k + m % 3)
        X, W = Rows(m, k, torch.float32, dx.ld, value=x), Rows(2 * n, k, torch.float32, dx.ld, value=w)
        P, D = Rows(m, 2 * n, torch.float32, value=pre), Rows(m, n, torch.float32, value=dh)
        p = mm.gated_params(0, m, n, k, gate=GATES[m % 2], ldx=dx.ld, ldw=dx.ld)
        mm.mm_gated_grad(p, X.buf, W.buf, P.buf, D.buf, dpre.buf, dx.buf, dw.buf, stream=stream())
        d = dpre.t.contiguous()
        same(dx.t, d, w.t().contiguous(), 2 * n, "dx")
        same(dw.t, d.t().contiguous(), x.t().contiguous(), m, "dw")


@pytest.mark.parametrize("m,n,k", F32_SHAPES)
def test_largest_numbers(m, n, k):
    """The largest numbers of f32, as masks hold them, among ordinary ones: finite sums stay finite."""
    top = torch.finfo(torch.float32).max
    x, w = randn(1, m, k), (randn(2, 2 * n, k) * 2.0 ** -14).clamp(-2.0 ** -13, 2.0 ** -13)
    x[::3, 0], x[1::3, k // 2], x[2::5, -1] = -top, top, -top
    for pad in ((4, 1) if k % 4 == 0 else (1,)):
        for a, b in ((x, w), (w[:1].expand(m, k).contiguous(), x[:1].expand(2 * n, k).contiguous())):
            want, absolute = products(a, b)
            near(forward(a, b, m, n, k, pad), want, bound(want, absolute, k), "pre")
