"""f32 products of the feed-forward block with operands far below 1: every form gives
sums in f32 down to the smallest numbers that f32 holds.

The bound is that of the other tests, (K + 8) U sum|x w| (the form in three bf16 parts
leaves out at most 2^-21 = 8 U of a product and rounds each sum a few times, f32
instructions round each product and each sum once), with U |sum| more for bits of
operands below 2^-133 that a form may leave where they are less than that, and half of
the smallest number, 2^-150, for each of the K + 8 roundings of sums below 2^-126."""
from __future__ import annotations

import pytest
import torch

import ffn_ref as ref
import gemv_expert_id_amd as mm
from ffn_ref import U
from test_gpu_ffn import F32_SHAPES, GATES, Rows, randn, stream

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def bound(want, absolute, terms):
    return (terms + 8) * U * absolute + U * want.abs() + (terms + 8) * 2.0 ** -150


def near(got, want, e, what):
    bad = ~((got.double() - want).abs() <= e)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / e)[bad].max()):.3g} of its bound"


def scaled(seed, rows, width, exponent):
    """Normal values times 2^exponent, which f32 rounds once where they fall below 2^-126."""
    return (randn(seed, rows, width).double() * 2.0 ** exponent).float()


def mixed(seed, rows, width, exponent):
    """Ordinary rows, rows of tiny values, ordinary rows with a few of them, zero rows, and single values."""
    x, tiny = randn(seed, rows, width), scaled(seed + 1, rows, width, exponent)
    kind = torch.arange(rows, device=DEV)[:, None] % 5
    some = torch.arange(width, device=DEV)[None] % 7 == 3
    x = torch.where(kind == 1, tiny, torch.where((kind == 2) & some, tiny, x))
    x = torch.where(kind == 3, torch.zeros_like(x), x)
    return torch.where(kind == 4, tiny * (torch.arange(width, device=DEV) == width - 1), x)


def products(x, w):
    x, w = x.double(), w.double()
    return x @ w.t(), x.abs() @ w.abs().t()


def check(x, w, m, n, k, pad):
    X, W = Rows(m, k, torch.float32, k + pad, value=x), Rows(2 * n, k, torch.float32, k + pad, value=w)
    h, pre = Rows(m, n, torch.float32), Rows(m, 2 * n, torch.float32)
    p = mm.gated_params(0, m, n, k, gate=GATES[m % 2], ldx=X.ld, ldw=W.ld)
    mm.mm_gated(p, X.buf, W.buf, h.buf, pre.buf, stream=stream())
    want, absolute = products(x, w)
    near(pre.t, want, bound(want, absolute, k), "pre")


SMALL = [(-112, 0), (-118, 0), (-125, 0), (-135, 20), (-145, 30), (0, -116), (-60, -60), (-70, -70), (-115, -20)]


@pytest.mark.parametrize("m,n,k", F32_SHAPES)
def test_small_rows(m, n, k):
    for i, (ex, ew) in enumerate(SMALL):
        for pad in ((4, 1) if k % 4 == 0 else (1,)):
            check(scaled(i, m, k, ex), scaled(i + 50, 2 * n, k, ew), m, n, k, pad)


@pytest.mark.parametrize("m,n,k", F32_SHAPES)
def test_small_among_ordinary(m, n, k):
    for pad in ((4, 1) if k % 4 == 0 else (1,)):
        check(mixed(1, m, k, -118), randn(3, 2 * n, k), m, n, k, pad)
        check(randn(4, m, k), mixed(5, 2 * n, k, -124), m, n, k, pad)
        check(mixed(6, m, k, -120), mixed(8, 2 * n, k, -112), m, n, k, pad)


# Rows, columns and contractions of every form of dx and dw, among them those that few rows over a long contraction take.
PRODUCTS = [(1, 511, 33), (1, 512, 1), (2, 513, 17), (16, 1040, 520), (17, 2047, 16), (32, 4111, 64), (40, 600, 6), (40, 600, 65), (70, 700, 700),
            (33, 300, 4099), (130, 1001, 500), (300, 130, 1030), (1024, 70, 67), (2001, 300, 500), (2100, 2, 3), (600, 9, 40), (1500, 700, 97)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("how", ["all", "mixed"])
def test_small_gradients(m, n, k, how):
    """dh, and so dpre, of tiny values; then tiny rows of x and w."""
    for e in (-110, -117, -124):
        made = scaled if how == "all" else mixed
        pre, dh = randn(1, m, 2 * n), made(2, m, n, e)
        for x, w in ((randn(4, m, k), randn(5, 2 * n, k)), (made(6, m, k, e + 8), made(8, 2 * n, k, e + 8))):
            if x[0, 0].abs() < 2.0 ** -90:
                dh = randn(9, m, n)
            dpre, dx, dw = Rows(m, 2 * n, torch.float32), Rows(m, k, torch.float32, k + m % 3), Rows(2 * n, k, torch.float32, k + m % 3)
            X, W = Rows(m, k, torch.float32, dx.ld, value=x), Rows(2 * n, k, torch.float32, dx.ld, value=w)
            P, D = Rows(m, 2 * n, torch.float32, value=pre), Rows(m, n, torch.float32, value=dh)
            p = mm.gated_params(0, m, n, k, gate=GATES[m % 2], ldx=dx.ld, ldw=dx.ld)
            mm.mm_gated_grad(p, X.buf, W.buf, P.buf, D.buf, dpre.buf, dx.buf, dw.buf, stream=stream())
            d = dpre.t
            assert bool(d.isfinite().all()) and bool((d != 0).any())
            want, absolute = products(d, w.t())
            near(dx.t, want, bound(want, absolute, 2 * n), f"dx, 2^{e}")
            want, absolute = products(d.t(), x.t())
            near(dw.t, want, bound(want, absolute, m), f"dw, 2^{e}")


@pytest.mark.parametrize("m,n,k", [s for s in F32_SHAPES if s[0] > 16])
def test_small_recomputed(m, n, k):
    """dpre from tiny pre-activations computed again: dh brings it back among ordinary numbers."""
    for pad in ((4, 1) if k % 4 == 0 else (1,)):
        x, w, dh = scaled(1, m, k, -119), randn(2, 2 * n, k), scaled(3, m, n, 60)
        X, W = Rows(m, k, torch.float32, k + pad, value=x), Rows(2 * n, k, torch.float32, k + pad, value=w)
        D, dpre = Rows(m, n, torch.float32, value=dh), Rows(m, 2 * n, torch.float32)
        p = mm.gated_params(0, m, n, k, gate=GATES[m % 2], ldx=X.ld, ldw=W.ld)
        mm.mm_gated_grad(p, X.buf, W.buf, None, D.buf, dpre.buf, None, None, stream=stream())
        pre, absolute = products(x, w)
        ep = bound(pre, absolute, k)
        want, e = ref.gated_grad(pre, ep, dh, GATES[m % 2])
        # of act(G), G tiny: its slope, 12 roundings (a sigmoid next to 1/2 and two products), and three below 2^-126
        e[:, n:] = dh.abs().double() * (ref.SLOPE * ep[:, :n] + 12 * U * ref.act(pre[:, :n], GATES[m % 2]).abs() + 3 * 2.0 ** -150)
        near(dpre.t, want, e + U * (want.abs() + e), "dpre")


def with_lost(t):
    """Values with bits below 2^-133 in every seventh row, one ordinary row of them."""
    t = t.clone()
    t[3::7] = scaled(77, *t.shape, -120)[3::7]
    t[4::14, -1] = 2.0 ** -130 + 2.0 ** -140
    return t


@pytest.mark.parametrize("m,n,k", F32_SHAPES)
def test_other_sums_keep_their_bits(m, n, k):
    """Sums whose own operands the parts hold, ordinary ones and small ones, do not change with other rows and columns."""
    for pad in ((4, 1) if k % 4 == 0 else (1,)):
        x, w = randn(1, m, k), randn(2, 2 * n, k)
        x[::2] *= 2.0 ** -103
        x[::2] = (x[::2].view(torch.int32) & ~0xFF).view(torch.float32)  # 16 bits, from 2^-118 on above 2^-133
        x[::2] = torch.where(x[::2].abs() < 2.0 ** -117, torch.zeros_like(x[::2]), x[::2])
        first = None
        for a, b in ((x, w), (with_lost(x), w), (x, with_lost(w))):
            X, W = Rows(m, k, torch.float32, k + pad, value=a), Rows(2 * n, k, torch.float32, k + pad, value=b)
            h, pre = Rows(m, n, torch.float32), Rows(m, 2 * n, torch.float32)
            mm.mm_gated(mm.gated_params(0, m, n, k, ldx=X.ld, ldw=W.ld), X.buf, W.buf, h.buf, pre.buf, stream=stream())
            first = pre.t if first is None else first
            kept = (a == x).all(1)[:, None] & (b == w).all(1)[None]
            assert torch.equal(pre.t[kept], first[kept]), "other sums have changed"


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_other_gradients_keep_their_bits(m, n, k):
    """As above for dx, by columns of w, and dw, by columns of x; a call gives the same bits again."""
    pre, dh, x, w = randn(1, m, 2 * n), randn(2, m, n) * 2.0 ** -99, randn(3, m, k), randn(4, 2 * n, k)
    outs = []
    for a, b in ((x, w), (with_lost(x.t()).t().contiguous(), with_lost(w.t()).t().contiguous())):
        for _ in range(2):
            dpre, dx, dw = Rows(m, 2 * n, torch.float32), Rows(m, k, torch.float32), Rows(2 * n, k, torch.float32)
            X, W = Rows(m, k, torch.float32, value=a), Rows(2 * n, k, torch.float32, value=b)
            P, D = Rows(m, 2 * n, torch.float32, value=pre), Rows(m, n, torch.float32, value=dh)
            mm.mm_gated_grad(mm.gated_params(0, m, n, k), X.buf, W.buf, P.buf, D.buf, dpre.buf, dx.buf, dw.buf, stream=stream())
            outs.append((dx.t, dw.t, (b == w).all(0), (a == x).all(0)))
    for i in range(0, 4, 2):
        assert torch.equal(outs[i][0], outs[i + 1][0]) and torch.equal(outs[i][1], outs[i + 1][1]), "differs from call to call"
    for i in (0, 1):
        kept = outs[2][2 + i]
        assert torch.equal(outs[0][i][:, kept], outs[2][i][:, kept]), "other columns have changed"
