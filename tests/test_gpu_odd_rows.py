"""16-bit products of operands whose rows have an odd length and a pitch of whole
16-byte pieces: the last element of the last row is alone in its four bytes, and every
kernel that takes such operands has to read it. Its factor and the one it meets are
large, so that their term alone is past the bound; what lies between rows is NaN."""
from __future__ import annotations

import pytest
import torch

import gemv_expert_id_amd as mm
from ffn_ref import TORCH, U, gated_grad, rounding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def operand(seed, rows, width, dtype, pad=0):
    """[rows, width] with a pitch of whole 16-byte pieces, NaN between rows; and its pitch and buffer."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ld = width + -width % 8 + pad
    store = torch.full((rows * ld + 16,), float("nan"), dtype=dtype, device=DEV)
    t = store.as_strided((rows, width), (ld, 1))
    t.copy_(torch.randn(rows, width, generator=g, device=DEV))
    return t, ld, mm.Buf(store.data_ptr(), ((rows - 1) * ld + width) * 2)


def near(got, want, absolute, terms, dt, what):
    """Sums of `terms` products in f32, rounded once."""
    e = (terms + 8) * U * absolute
    err, bound = (got.double() - want).abs(), e + rounding(dt, want.abs() + e)
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{what}: {bad.nonzero()[:4].tolist()} of {tuple(got.shape)}, {float((err / bound)[bad].max()):.3g} of the bound"


REACHED = set()
GEMMS = [(130, 201, 33), (70, 300, 127), (301, 135, 257), (257, 300, 1001),  # tiles staged through registers
         (129, 131, 256), (1023, 1025, 512),                                 # 128 x 128 tiles by DMA
         (3585, 3457, 256), (4095, 4095, 256)]                               # 256 x 256 tiles by DMA


@pytest.mark.parametrize("dt", [1, 2])
@pytest.mark.parametrize("ta", [False, True])
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("m,n,k", GEMMS)
def test_gemm(dt, ta, tb, m, n, k):
    a, lda, abuf = operand(m, *((k, m) if ta else (m, k)), TORCH[dt])
    b, ldb, bbuf = operand(n + 1, *((n, k) if tb else (k, n)), TORCH[dt])
    a[-1, -1], b[-1, -1] = 30, 40
    c, ldc, cbuf = operand(1, m, n, TORCH[dt])
    A, B = a.double().t() if ta else a.double(), b.double().t() if tb else b.double()
    A, B = A.contiguous(), B.contiguous()
    rec = mm.mm_gemm(mm.gemm_desc(dt, m, n, k, trans_a=ta, trans_b=tb, lda=lda, ldb=ldb, ldc=ldc), abuf, bbuf, cbuf,
                     stream=torch.cuda.current_stream())
    near(c, A @ B, A.abs() @ B.abs(), k, dt, f"kernel {rec.kernel} {rec.variant}")
    REACHED.add((rec.kernel, rec.variant // 2 * 2))


@pytest.mark.parametrize("ta,tb", [(False, False), (True, False), (True, True)])
def test_batch(ta, tb):
    """Every matrix of a batch ends so."""
    m, n, k, count = 131, 133, 129 if not ta else 256, 3
    made = [(operand(i, *((k, m) if ta else (m, k)), TORCH[2]), operand(9 + i, *((n, k) if tb else (k, n)), TORCH[2])) for i in range(count)]
    for (a, _, _), (b, _, _) in made:
        a[-1, -1], b[-1, -1] = 30, 40
    lda, ldb = made[0][0][1], made[0][1][1]
    join = lambda ts, ld: torch.stack([torch.nn.functional.pad(t, (0, ld - t.shape[1]), value=float("nan")) for t in ts])  # noqa: E731
    A, B = join([x[0][0] for x in made], lda), join([x[1][0] for x in made], ldb)
    c = torch.zeros(count, m, n, dtype=TORCH[2], device=DEV)
    mm.mm_gemm(mm.gemm_desc(2, m, n, k, batch=count, trans_a=ta, trans_b=tb, lda=lda, ldb=ldb, stride_a=A[0].numel(),
                            stride_b=B[0].numel()), mm.buf(A), mm.buf(B), mm.buf(c), stream=torch.cuda.current_stream())
    for i, ((a, _, _), (b, _, _)) in enumerate(made):
        x, y = a.double().t() if ta else a.double(), b.double().t() if tb else b.double()
        x, y = x.contiguous(), y.contiguous()
        near(c[i], x @ y, x.abs() @ y.abs(), k, 2, f"matrix {i}")


def test_every_tile_was_reached():
    if len(REACHED) > 1:  # (with the tests above)
        assert REACHED == {(mm.MM_KERNEL_GEMM_TILED, 0), (mm.MM_KERNEL_GEMM_LARGE, 128), (mm.MM_KERNEL_GEMM_LARGE, 256)}


# Rows of x and w (and of dx and dw) odd: dx = dpre . w and dw = dpre^T . x end in column k - 1, in the GEMM and in the
# forms of the feed-forward products, on either side of the choice.
@pytest.mark.parametrize("dt", [1, 2])
@pytest.mark.parametrize("m,n,k,pad", [(2048, 1024, 2047, 0), (2048, 1024, 2047, 8), (1024, 1024, 4095, 0), (4001, 1024, 4095, 0),
                                       (900, 1000, 1537, 0), (1000, 900, 2045, 0), (300, 520, 1409, 16), (130, 64, 33, 0)])
def test_gated_gradients(dt, m, n, k, pad):
    t = TORCH[dt]
    x, ldx, xbuf = operand(1, m, k, t, pad)
    w, ldw, wbuf = operand(2, 2 * n, k, t, pad)
    pre, _, prebuf = operand(3, m, 2 * n, t)
    dh, _, dhbuf = operand(4, m, n, t)
    pre[-1, -1], pre[-1, n - 1], dh[-1, -1] = 4, 4, 4  # the last pre-activations have large gradients
    x[-1, -1], w[-1, -1] = 40, 40
    dpre, _, dprebuf = operand(5, m, 2 * n, t)
    dx, _, dxbuf = operand(6, m, k, t, pad)
    dw, _, dwbuf = operand(7, 2 * n, k, t, pad)
    mm.mm_gated_grad(mm.gated_params(dt, m, n, k, ldx=ldx, ldw=ldw, ldpre=pre.stride(0), ldh=dh.stride(0)), xbuf, wbuf, prebuf,
                     dhbuf, dprebuf, dxbuf, dwbuf, stream=torch.cuda.current_stream())
    want, e = gated_grad(pre.double(), torch.zeros(m, 2 * n, dtype=torch.float64, device=DEV), dh, 1)
    assert bool(((dpre.double() - want).abs() <= e + rounding(dt, want.abs() + e)).all())
    d, X, W = dpre.double(), x.double(), w.double()
    near(dx, d @ W, d.abs() @ W.abs(), 2 * n, dt, "dx")
    d = d.t().contiguous()
    near(dw, d @ X, d.abs() @ X.abs(), m, dt, "dw")
