"""GPU tests of the feed-forward block's operators against the 64-bit definitions
in ffn_ref.py, with the error bounds derived there plus half a step of the output's
type. Whole numbers have to be equal. Memory around every operand holds NaN (or a
code that would show), memory around every output a sentinel that must survive."""
from __future__ import annotations

import pytest
import torch

import ffn_ref as ref
import gemv_expert_id_amd as mm
from ffn_ref import TORCH, rounding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = [0, 1, 2]
GATES = [ref.SILU, ref.GELU]


def stream():
    return torch.cuda.current_stream()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(seed, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen(seed), device=DEV) * scale).to(dtype)


class Rows:
    """[rows, width] on the GPU with a pitch, `shift` elements into memory filled with `fill`."""

    def __init__(self, rows, width, dtype, ld=0, shift=0, value=None, fill=None):
        self.rows, self.width, self.ld, self.shift = rows, width, ld or width, shift
        self.fill = fill if fill is not None else (float("nan") if dtype.is_floating_point else 99)
        self.store = torch.full((shift + rows * self.ld + 16,), self.fill, dtype=dtype, device=DEV)
        self.t = self.store[shift:].as_strided((rows, width), (self.ld, 1))
        if value is not None:
            self.t.copy_(value)

    @property
    def buf(self):
        z = self.store.element_size()
        return mm.Buf(self.store.data_ptr() + self.shift * z, ((self.rows - 1) * self.ld + self.width) * z)

    def untouched(self):
        """Everything outside the tensor still holds the fill."""
        probe = self.store.clone()
        probe[self.shift:].as_strided((self.rows, self.width), (self.ld, 1)).fill_(self.fill)
        same = probe.isnan() if self.fill != self.fill else probe == self.fill
        assert bool(same.all()), "written outside the output"


def near(got, want, bound, what):
    assert got.shape == want.shape
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound)[bad].max()):.3g} of its bound"


# ---- the gated block -------------------------------------------------------------


def gated_operands(dt, m, n, k, pad, shift):
    t = TORCH[dt]
    x = Rows(m, k, t, k + pad, shift, randn(m + n, m, k))
    w = Rows(2 * n, k, t, k + pad, shift, randn(n + k, 2 * n, k, scale=1.5 / k ** 0.5))
    return x, w


def check_gated(dt, m, n, k, gate=ref.SILU, saved=True, pad=0, shift=0):
    t = TORCH[dt]
    x, w = gated_operands(dt, m, n, k, pad, shift)
    h = Rows(m, n, t, n + pad, shift)
    pre = Rows(m, 2 * n, t, 2 * n + pad, shift) if saved else None
    p = mm.gated_params(dt, m, n, k, gate=gate, ldx=x.ld, ldw=w.ld, ldpre=pre.ld if saved else 0, ldh=h.ld)
    rec = mm.mm_gated(p, x.buf, w.buf, h.buf, pre.buf if saved else None, stream=stream())
    assert rec.kernel == mm.MM_KERNEL_GATED and rec.route == mm.MM_ROUTE_GATED and rec.dispatch_count == 1
    want, wpre, e, epre = ref.gated(x.t, w.t, gate)
    near(h.t, want, e + rounding(dt, want.abs() + e), "h")
    h.untouched()
    if saved:
        near(pre.t, wpre, epre + rounding(dt, wpre.abs() + epre), "pre")
        pre.untouched()
    return rec


def check_grad(dt, m, n, k, gate=ref.SILU, saved=True, pad=0, shift=0, want=("dx", "dw"), in_place=False):
    t = TORCH[dt]
    x, w = gated_operands(dt, m, n, k, pad, shift)
    dh = Rows(m, n, t, n + pad, shift, randn(7, m, n))
    _, pre, _, e = ref.gated(x.t, w.t, gate)
    dpre = Rows(m, 2 * n, t, 2 * n + pad, shift)
    held = None
    if saved:
        held = dpre if in_place else Rows(m, 2 * n, t, 2 * n + pad, shift)
        held.t.copy_(pre)
        pre, e = held.t.double().clone(), torch.zeros_like(pre)
    dx = Rows(m, k, t, k + pad, shift) if "dx" in want else None
    dw = Rows(2 * n, k, t, k + pad, shift) if "dw" in want else None
    p = mm.gated_params(dt, m, n, k, gate=gate, ldx=x.ld, ldw=w.ld, ldpre=dpre.ld, ldh=dh.ld)
    rec = mm.mm_gated_grad(p, x.buf, w.buf, held.buf if saved else None, dh.buf, dpre.buf,
                           dx.buf if dx else None, dw.buf if dw else None, stream=stream())
    assert rec.route == mm.MM_ROUTE_GATED and rec.dispatch_count == 1 + len(want)
    wd, ed = ref.gated_grad(pre, e, dh.t, gate)
    near(dpre.t, wd, ed + rounding(dt, wd.abs() + ed), "dpre")
    dpre.untouched()
    if dx:  # of the rounded dpre
        v, ev = ref.products(dpre.t, w.t.t())
        near(dx.t, v, ev + rounding(dt, v.abs() + ev), "dx")
        dx.untouched()
    if dw:
        v, ev = ref.products(dpre.t.t(), x.t.t())
        near(dw.t, v, ev + rounding(dt, v.abs() + ev), "dw")
        dw.untouched()
    return rec


SIZES = [(1, 1, 1), (1, 64, 64), (2, 3, 5), (5, 17, 24), (16, 16, 32), (17, 33, 40), (33, 130, 72), (64, 64, 128),
         (65, 127, 264), (129, 65, 200), (130, 192, 513), (300, 257, 96)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated(dt, m, n, k):
    check_gated(dt, m, n, k, gate=GATES[(m + n) % 2], saved=n % 2 == 1)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (3, 5), (8, 8)])
@pytest.mark.parametrize("m", [3, 70])
def test_gated_pitches_and_starts(dt, pad, shift, m):
    check_gated(dt, m, 50, 88, gate=ref.GELU, pad=pad, shift=shift)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("saved", [False, True])
def test_gated_grad(dt, m, n, k, saved):
    check_grad(dt, m, n, k, gate=GATES[(m + n) % 2], saved=saved)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (3, 5), (8, 8)])
@pytest.mark.parametrize("saved", [False, True])
def test_gated_grad_pitches_and_starts(dt, pad, shift, saved):
    check_grad(dt, 37, 50, 88, gate=ref.GELU, saved=saved, pad=pad, shift=shift)


@pytest.mark.parametrize("want", [(), ("dx",), ("dw",)])
@pytest.mark.parametrize("saved", [False, True])
def test_gated_grad_parts(want, saved):
    check_grad(2, 40, 48, 64, saved=saved, want=want)


@pytest.mark.parametrize("dt", DTYPES)
def test_gated_grad_in_place(dt):
    check_grad(dt, 41, 50, 64, in_place=True)
    check_grad(dt, 41, 51, 64, in_place=True, pad=3, shift=1)


@pytest.mark.parametrize("gate", GATES)
def test_gradients_against_differences(gate):
    """f32 gradients against differences of the 64-bit forward; the difference's own error is step^2."""
    m, n, k = 4, 6, 8
    x, w, dh = randn(1, m, k), randn(2, 2 * n, k, scale=0.5), randn(3, m, n)
    dpre, dx, dw = (torch.empty(*s, device=DEV) for s in ((m, 2 * n), (m, k), (2 * n, k)))
    mm.mm_gated_grad(mm.gated_params(0, m, n, k, gate=gate), mm.buf(x), mm.buf(w), None, mm.buf(dh), mm.buf(dpre),
                     mm.buf(dx), mm.buf(dw), stream=stream())
    f = lambda x, w: float((ref.gated(x, w, gate)[0] * dh.double()).sum())  # noqa: E731
    step = 1e-5
    for t, grad in ((x.double(), dx), (w.double(), dw)):
        for i in range(0, t.numel(), 5):
            up, down = t.clone(), t.clone()
            up.view(-1)[i] += step
            down.view(-1)[i] -= step
            pair = (up, down) if grad is dw else (up, down)
            diff = (f(x.double(), pair[0]) - f(x.double(), pair[1]) if grad is dw else
                    f(pair[0], w.double()) - f(pair[1], w.double())) / (2 * step)
            assert abs(diff - float(grad.view(-1)[i])) < 2e-5


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("gate", GATES)
def test_far_pre_activations(dt, gate):
    """Gates far on both sides, zeros, and values whose cubes leave f32: no NaN, h and gradients as defined."""
    t = TORCH[dt]
    big = 3e4 if dt == 1 else 1e18
    g = torch.tensor([0.0, -0.0, 1.0, -1.0, 30.0, -30.0, 80.0, -80.0, 1000.0, -1000.0, big, -big], device=DEV)
    n = g.numel()
    pre = torch.cat((g, torch.ones(n, device=DEV))).to(t)[None].contiguous()
    dh = torch.full((1, n), 0.5, dtype=t, device=DEV)
    x, w = torch.ones(1, 1, dtype=t, device=DEV), pre.t().contiguous()
    p = mm.gated_params(dt, 1, n, 1, gate=gate)
    h, dpre = torch.empty(1, n, dtype=t, device=DEV), torch.empty(1, 2 * n, dtype=t, device=DEV)
    mm.mm_gated(p, mm.buf(x), mm.buf(w), mm.buf(h), None, stream=stream())
    want, _, e, _ = ref.gated(x, w, gate)
    near(h, want, e + rounding(dt, want.abs() + e), "h")
    wd, ed = ref.gated_grad(pre.double(), torch.zeros(1, 2 * n, dtype=torch.float64, device=DEV), dh, gate)
    for saved in (mm.buf(pre), None):
        mm.mm_gated_grad(p, mm.buf(x), mm.buf(w), saved, mm.buf(dh), mm.buf(dpre), None, None, stream=stream())
        # x w here is one product of numbers with few bits: exact
        near(dpre, wd, ed + rounding(dt, wd.abs() + ed), "dpre")


# ---- codes -----------------------------------------------------------------------


def check_quant(dt, m, k, ldx=0, ldq=0, shift=0, value=None):
    x = Rows(m, k, TORCH[dt], ldx, shift, randn(m * 31 + k, m, k) if value is None else value)
    q, s = Rows(m, k, torch.int8, ldq, shift), Rows(m, 1, torch.float32, 0, shift % 4)
    rec = mm.mm_i8_quant(mm.quant_params(dt, m, k, ldx=x.ld, ldq=q.ld), x.buf, q.buf, s.buf, stream=stream())
    assert rec.kernel == mm.MM_KERNEL_I8_QUANT and rec.route == mm.MM_ROUTE_I8 and rec.dispatch_count == 1
    wq, ws = ref.quantise(x.t)
    assert torch.equal(s.t[:, 0], ws)
    assert torch.equal(q.t, wq), f"{int((q.t != wq).sum())} codes differ"
    q.untouched()
    s.untouched()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,k", [(1, 1), (1, 7), (3, 16), (2, 255), (5, 256), (4, 1000), (7, 2048), (2, 4097), (1, 8192),
                                 (3, 11008), (2, 16385), (1, 40000), (1, 100003), (600, 64), (2100, 33), (1500, 520)])
def test_quant(dt, m, k):
    check_quant(dt, m, k)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("ldx,ldq,shift", [(1030, 1031, 0), (1024, 1024, 1), (1025, 1040, 3), (1032, 1024, 8), (1024, 1025, 0)])
@pytest.mark.parametrize("m", [3, 1100])
def test_quant_pitches_and_starts(dt, ldx, ldq, shift, m):
    check_quant(dt, m, 1023 if ldx == 1025 else 1024, ldx, ldq, shift)


@pytest.mark.parametrize("dt", DTYPES)
def test_quant_ties_and_every_value(dt):
    """Exact halves of a scale, zero rows, rows of tiny numbers; in 16 bits every finite value."""
    half = torch.arange(-254, 255, device=DEV).float() / 2
    rows = [half * f for f in (1.0, 0.25, 2.0 ** -8, 0.0)]
    if dt != 1:
        rows += [half * 2.0 ** -120, half * 2.0 ** -128, half * 2.0 ** -133]
    check_quant(dt, len(rows), 509, value=torch.stack(rows))
    if dt:
        bits = torch.arange(-32768, 32768, dtype=torch.int32, device=DEV).to(torch.int16).view(TORCH[dt])
        v = bits[torch.isfinite(bits)]
        check_quant(dt, 1, v.numel(), value=v[None])
        v = v[v.abs() < 100]
        check_quant(dt, 1, v.numel(), value=v[None])


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("k", [40, 5000, 70000])
def test_quant_rows_that_are_not_finite(dt, k):
    x = randn(5, 6, k, dtype=TORCH[dt])
    x[1, k // 2] = float("nan")
    x[2, k - 1] = float("inf")
    x[3, 0] = float("-inf")
    x[4, 1], x[4, k - 2] = float("inf"), float("nan")
    q, s = torch.full((6, k), 99, dtype=torch.int8, device=DEV), torch.zeros(6, device=DEV)
    mm.mm_i8_quant(mm.quant_params(dt, 6, k), mm.buf(x), mm.buf(q), mm.buf(s), stream=stream())
    wq, ws = ref.quantise(x[[0, 5]])
    assert torch.equal(q[[0, 5]], wq) and torch.equal(s[[0, 5]], ws)
    assert not q[1:5].any()
    assert bool(s[[1, 4]].isnan().all()) and bool(torch.isposinf(s[[2, 3]]).all())
    w, ws, y = torch.ones(3, 48, dtype=torch.int8, device=DEV), torch.ones(3, device=DEV), torch.zeros(6, 3, device=DEV)
    qx = torch.zeros(6, 48, dtype=torch.int8, device=DEV)
    qx[:, :40] = q[:, :40]
    mm.mm_i8_gemm(mm.i8_params(0, 6, 3, 48), mm.buf(qx), mm.buf(s), mm.buf(w), mm.buf(ws), mm.buf(y), stream=stream())
    assert bool(y[1:5].isnan().all()) and bool(torch.isfinite(y[[0, 5]]).all())


def codes(seed, m, k, low=-127):
    return torch.randint(low, 128, (m, k), generator=gen(seed), device=DEV, dtype=torch.int8)


def check_i8(dt, m, n, k, gate=ref.NONE, pad=0, ypad=0, shift=0, low=-127):
    rows = n * (1 + (gate > 0))
    x = Rows(m, k, torch.int8, k + pad, shift, codes(m + k, m, k, low))
    w = Rows(rows, k, torch.int8, k + pad, shift, codes(n + k, rows, k, low))
    s = Rows(m, 1, torch.float32, 0, shift % 4, torch.rand(m, 1, generator=gen(1), device=DEV) * 0.02 + 1e-3)
    ws = Rows(rows, 1, torch.float32, 0, shift % 3, (torch.rand(rows, 1, generator=gen(2), device=DEV) + 0.1) / (40 * k ** 0.5))
    y = Rows(m, n, TORCH[dt], n + ypad, shift % 16)
    p = mm.i8_params(dt, m, n, k, gate=gate, ldx=x.ld, ldw=w.ld, ldy=y.ld)
    rec = mm.mm_i8_gemm(p, x.buf, s.buf, w.buf, ws.buf, y.buf, stream=stream())
    assert rec.kernel == mm.MM_KERNEL_I8 and rec.route == mm.MM_ROUTE_I8 and rec.dispatch_count == 1
    want, e = ref.i8(x.t, s.t[:, 0], w.t, ws.t[:, 0], gate)
    near(y.t, want, e + rounding(dt, want.abs() + e), "y")
    y.untouched()
    return rec


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 64, 64), (1, 100, 4096), (2, 3, 48), (4, 300, 1040), (5, 17, 80), (8, 33, 2048),
                                   (16, 16, 128), (17, 33, 144), (33, 130, 208), (64, 64, 1024), (65, 127, 272),
                                   (129, 65, 4112), (130, 192, 528), (300, 257, 96)])
@pytest.mark.parametrize("gate", [ref.NONE, ref.SILU])
def test_i8(dt, m, n, k, gate):
    check_i8(dt, m, n, k, gate=gate)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("pad,ypad,shift", [(16, 1, 0), (0, 0, 16), (48, 3, 32), (16, 8, 48)])
@pytest.mark.parametrize("m", [1, 3, 70, 200])
@pytest.mark.parametrize("gate", [ref.NONE, ref.GELU])
def test_i8_pitches_and_starts(dt, pad, ypad, shift, m, gate):
    check_i8(dt, m, 50, 176, gate=gate, pad=pad, ypad=ypad, shift=shift)


@pytest.mark.parametrize("m,n", [(1, 33), (9, 40), (70, 130)])
def test_i8_largest_sums(m, n):
    """The longest contraction with every code -128: sums of almost 2^31, exact."""
    k = mm.MM_I8_MAX_K
    x, w = (torch.full((r, k), -128, dtype=torch.int8, device=DEV) for r in (m, n))
    s, ws, y = torch.ones(m, device=DEV), torch.ones(n, device=DEV), torch.empty(m, n, device=DEV)
    mm.mm_i8_gemm(mm.i8_params(0, m, n, k), mm.buf(x), mm.buf(s), mm.buf(w), mm.buf(ws), mm.buf(y), stream=stream())
    assert bool((y == float(k * 16384)).all())  # 8191 * 2^18: 13 bits
    check_i8(0, m, n, k, low=-128)
    check_i8(2, m, n, 4096, gate=ref.SILU, low=-128)


# ---- the forms a product takes, by its size ------------------------------------------


TILES = [(16, 16, 0, 0, 0), (32, 16, 512, 0.257, 0.60), (64, 64, 256, 0.300, 1.93), (64, 128, 256, 0.320, 2.26),
         (128, 128, 256, 0.607, 2.15), (256, 128, 256, 0.956, 3.35), (256, 256, 256, 1.593, 7.15)]


def form(m, rows, row_bytes):
    """The form that the measured costs choose, as a receipt's variant."""
    up = lambda a, b: -(-a // b)  # noqa: E731

    def cost(f):
        tiles, one = up(m, f[0]) * up(rows, f[1]), up(row_bytes, 128) * f[3] + f[4]
        us = up(tiles, f[2]) * one
        if f is TILES[-1] and 0 < tiles % f[2] <= f[2] // 2:  # a last round of halves
            us -= one - (up(row_bytes, 128) * TILES[-2][3] + TILES[-2][4])
        return us

    f = min(TILES[1:], key=cost) if m > 16 else TILES[0]
    return f[0] + 4096 * f[1]


# m, n, k of a gated product in 16 bits (k twice as long in codes); every form is among them
SHAPES = [(1, 8209, 520), (16, 8209, 1032), (1, 70, 4104), (9, 33, 8), (17, 145, 1048), (30, 257, 2048), (40, 33, 1032),
          (33, 4105, 264), (48, 8209, 520), (64, 1100, 8), (65, 1100, 1032), (200, 257, 72), (300, 1411, 520), (500, 1411, 2056),
          (129, 8209, 264), (1100, 1985, 200), (700, 2049, 1032), (1200, 4097, 520), (3500, 1795, 200), (3329, 1985, 1096), (4200, 2400, 136), (4100, 2700, 264)]


def test_every_form_is_reached():
    assert {form(m, 2 * n, 2 * k) for m, n, k in SHAPES} == {f[0] + 4096 * f[1] for f in TILES}


@pytest.mark.parametrize("dt", [1, 2])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gated_forms(dt, m, n, k):
    assert check_gated(dt, m, n, k, gate=GATES[m % 2], saved=n % 2 == 1, pad=8).variant == form(m, 2 * n, 2 * k)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_i8_forms(m, n, k):
    k = k // 8 * 16
    assert check_i8(m % 3, m, n, k, gate=GATES[m % 2], pad=16).variant == form(m, 2 * n, k)
    assert check_i8(m % 3, m, 2 * n - 1, k, pad=16).variant == form(m, 2 * n - 1, k)


# Contractions (2n) long enough for few rows to be split over a block's waves, and the borders of that.
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 511, 33), (1, 512, 1), (2, 513, 17), (16, 515, 49), (17, 2047, 16), (16, 1040, 4096),
                                   (13, 529, 4097), (17, 4096, 31), (32, 4111, 64), (33, 4111, 20)])
def test_long_contractions(dt, m, n, k):
    check_grad(dt, m, n, k, gate=GATES[m % 2], pad=n % 2, shift=k % 3, want=("dx",))


# Few tokens: 4 or 8 stages of 256 bytes ahead, by their number (here in bytes of k).
@pytest.mark.parametrize("row_bytes", [31 * 256, 32 * 256, 32 * 256 + 16, 33 * 256, 38 * 256 - 16, 40 * 256, 85 * 256 + 240, 96 * 256])
@pytest.mark.parametrize("m,n", [(1, 33), (16, 8), (30, 70)])
def test_stages(m, n, row_bytes):
    for dt in DTYPES:
        check_gated(dt, m, n, row_bytes // (2 if dt else 4), pad=8)
    check_i8(m % 3, m, n, row_bytes, gate=ref.SILU)
    check_i8(m % 3, m, 2 * n - 1, row_bytes, pad=16)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gradient_forms(m, n, k):
    assert check_grad(1, m, n, k, gate=GATES[m % 2], saved=False, want=()).variant == form(m, 2 * n, 2 * k)


@pytest.mark.parametrize("m,n,k", [(5, 4105, 264), (64, 8209, 72), (40, 70, 1032), (200, 257, 68), (1100, 1985, 200)])
def test_gated_forms_f32(m, n, k):
    check_gated(0, m, n, k, gate=GATES[m % 2], pad=4)
    check_grad(0, m, n, k, gate=GATES[m % 2], saved=False, want=())

# Products of f32 gradients: 16, 32 and 64 rows at a time, columns that no four fill, fewer than four of them, contractions
# that end inside a step.
@pytest.mark.parametrize("m,n,k", [(1, 33, 3), (3, 520, 5), (40, 600, 6), (40, 600, 65), (70, 700, 700), (33, 300, 4099), (130, 1001, 500), (200, 1500, 130),
                                   (300, 130, 1030), (1024, 70, 67), (1029, 250, 301), (2001, 300, 500), (2100, 2, 3), (2100, 1, 70), (600, 9, 40), (1500, 700, 97)])
def test_f32_gradients(m, n, k):
    check_grad(0, m, n, k, gate=GATES[m % 2], pad=m % 3, shift=n % 2)


def f32_form(m, n, k, chunked):
    """The choice among f32's forms, from their measured costs."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    cost = lambda bm, bn, kt, slots, step, start: up(up(m, bm) * up(2 * n, bn), slots) * (up(k, kt) * step + start)  # noqa: E731
    costs = {"waves 32 x 32": cost(32, 32, 256, 256, 1.78, 0.8), "waves 32 x 64": cost(32, 64, 256, 256, 2.55, 2.0),
             "waves 64 x 64": cost(64, 64, 128, 256, 1.6, 4.0), "128 x 128": cost(128, 128, 32, 512, 2.6, 14.0),
             "pipe" if chunked else "64 x 64": cost(64, 64, 32, 512, *((0.9, 1.0) if chunked else (1.2, 3.0)))}
    if chunked:
        if up(m, 64) * up(2 * n, 128) > 256:
            costs["broad"] = cost(64, 128, 32, 256, 0.74, 2.0)
        costs["thin"] = 0 if m <= 16 else cost(32, 16, 64, 256, 0.2, 0.5)
    return min(costs, key=costs.get)


F32_SHAPES = [(16, 300, 200), (17, 130, 64), (141, 149, 952), (70, 40, 8), (99, 902, 224), (69, 2185, 196), (67, 3656, 196),
              (70, 4105, 260), (300, 1409, 72), (513, 1411, 40), (1037, 2900, 300), (904, 3401, 520), (280, 3271, 204), (129, 4100, 130), (257, 2050, 131), (700, 4100, 33),
              (129, 90, 31), (65, 33, 1), (1100, 1985, 203)]


def test_every_f32_form_is_reached():
    assert {f32_form(*s, True) for s in F32_SHAPES if s[2] % 4 == 0} == {"thin", "waves 32 x 32", "waves 32 x 64", "waves 64 x 64", "128 x 128", "pipe", "broad"}
    assert {f32_form(*s, False) for s in F32_SHAPES} == {"waves 32 x 32", "waves 32 x 64", "waves 64 x 64", "128 x 128", "64 x 64"}


@pytest.mark.parametrize("m,n,k", F32_SHAPES)
def test_f32_forms(m, n, k):
    variant = {"thin": (16 if m <= 16 else 32) + 4096 * 16, "pipe": 64 + 4096 * 64, "broad": 64 + 4096 * 128}
    if k % 4 == 0:
        want = variant.get(f32_form(m, n, k, True), 0)
        assert check_gated(0, m, n, k, gate=GATES[m % 2], pad=4).variant == want
        assert check_grad(0, m, n, k, gate=GATES[m % 2], saved=False, want=()).variant == want
    assert check_gated(0, m, n, k, gate=GATES[m % 2], saved=n % 2 == 1, pad=1).variant == 0
    assert check_grad(0, m, n, k, gate=GATES[m % 2], saved=False, pad=3, shift=1, want=()).variant == 0


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 64, 96), (2, 128, 256), (37, 64, 96), (129, 128, 512), (300, 260, 264), (511, 192, 2040),
                                   (1025, 516, 72), (2, 4096, 2048), (700, 1024, 1032)])
def test_gradient_products(dt, m, n, k):
    """Rows of whole 16-byte pieces; contractions over tokens of any count."""
    check_grad(dt, m, n, k, gate=GATES[m % 2], pad=8)
    check_grad(dt, m, n, k, gate=GATES[m % 2], pad=0)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1100, 1985, 33), (1203, 1950, 129), (33, 1985, 1100), (1985, 70, 1985)])
def test_any_alignment_large_tiles(dt, m, n, k):
    check_gated(dt, m, n, k, pad=1)
    check_grad(dt, m, n, k, pad=1, saved=False)
    check_grad(dt, m, n, k, gate=ref.GELU)


# ---- far offsets ------------------------------------------------------------------
# Rows so far apart that the last ones lie past 2^32 bytes: just inside the pitches of the pipelined forms (below 4 MiB), and
# beyond them.


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("pitch,m,n,k", [((1 << 22) - 16, 1050, 530, 72), (1 << 24, 270, 140, 40), ((1 << 24) + 12, 265, 135, 33)])
def test_far_rows(dt, pitch, m, n, k):
    z = torch.finfo(TORCH[dt]).bits // 8
    check_gated(dt, m, n, k, pad=pitch // z - k)
    torch.cuda.empty_cache()
    check_grad(dt, m, n, k, pad=pitch // z - 2 * n, want=("dx",))
    torch.cuda.empty_cache()
    check_grad(dt, m, n, k, pad=pitch // z - 2 * n, saved=False, want=("dw",))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", DTYPES)
def test_far_rows_few(dt):
    z = torch.finfo(TORCH[dt]).bits // 8
    check_gated(dt, 9, 530, 72, pad=((1 << 22) - 16) // z - 72)  # few tokens
    check_grad(dt, 9, 530, 33, pad=(1 << 22) // z, want=("dx",))  # a contraction split over waves
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", DTYPES)
def test_far_codes(dt):
    z = torch.finfo(TORCH[dt]).bits // 8
    check_quant(dt, 270, 1000, ldx=(1 << 24) // z, ldq=(1 << 24) + 5)
    check_i8(dt, 1050, 1060, 80, pad=(1 << 22) - 96, ypad=(1 << 22) // z)
    torch.cuda.empty_cache()


# ---- values that are not finite ------------------------------------------------------


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k,pad", [(9, 40, 72, 8), (70, 70, 264, 8), (70, 70, 264, 1), (200, 600, 700, 4), (67, 3656, 196, 4), (300, 1409, 72, 8),
                                       (513, 1411, 40, 1), (1037, 2900, 300, 4)])
def test_rows_that_are_not_finite(dt, m, n, k, pad):
    """A NaN or an infinity stays in its token's row and in its weight's column."""
    t = TORCH[dt]
    x, w = gated_operands(dt, m, n, k, pad, 0)
    x.t[3, k // 2] = float("nan")
    x.t[m - 1, 0] = float("inf")
    w.t[5, k - 1] = float("nan")
    h, pre = Rows(m, n, t, n), Rows(m, 2 * n, t, 2 * n)
    mm.mm_gated(mm.gated_params(dt, m, n, k, ldx=x.ld, ldw=w.ld), x.buf, w.buf, h.buf, pre.buf, stream=stream())
    token = torch.zeros(m, 1, dtype=torch.bool, device=DEV)
    token[3] = token[m - 1] = True
    column = torch.zeros(1, 2 * n, dtype=torch.bool, device=DEV)
    column[0, 5] = True
    assert torch.equal(~pre.t.isfinite(), token | column)
    assert torch.equal(~h.t.isfinite(), token | column[:, :n])


def test_gradient_rows_that_are_not_finite():
    """dx: a token's row alone; dw: a pre-activation's row alone."""
    for dt, m, n, k in ((0, 70, 40, 60), (0, 20, 700, 40), (0, 300, 130, 257), (0, 1030, 70, 130), (1, 70, 40, 60), (2, 300, 192, 264), (2, 20, 700, 40)):
        t = TORCH[dt]
        x, w = gated_operands(dt, m, n, k, 0, 0)
        pre, dh = Rows(m, 2 * n, t, 2 * n, value=randn(1, m, 2 * n)), Rows(m, n, t, n, value=randn(2, m, n))
        dh.t[7, 2] = float("nan")
        dpre, dx, dw = Rows(m, 2 * n, t, 2 * n), Rows(m, k, t, k), Rows(2 * n, k, t, k)
        mm.mm_gated_grad(mm.gated_params(dt, m, n, k), x.buf, w.buf, pre.buf, dh.buf, dpre.buf, dx.buf, dw.buf, stream=stream())
        for got, rows in ((dx.t, [7]), (dw.t, [2, n + 2])):
            want = torch.zeros(got.shape[0], 1, dtype=torch.bool, device=DEV)
            want[rows] = True
            assert torch.equal(got.isnan(), want.expand_as(got))
