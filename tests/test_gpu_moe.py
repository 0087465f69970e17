"""GPU tests of the router, the sorted rows and the 4-bit products against the
64-bit definitions in moe_ref.py.

Tolerances: outputs of 16 bits are off by half a step of their value on top of
the error of the 32-bit sums, which is counted per addition (2^-24 of the
magnitude added). What is moved or counted has to be equal.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemv_expert_id_amd as mm
import moe_ref as ref
from moe_ref import NONE, TORCH, U, rounding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = [0, 1, 2]


def stream():
    return torch.cuda.current_stream()


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Padded:
    """A [rows, width] device tensor with a row pitch and a start that is only
    element-aligned, inside memory filled with a sentinel."""

    def __init__(self, rows, width, dtype, ld=0, shift=0, value=None):
        self.rows, self.width, self.ld, self.shift = rows, width, ld or width, shift
        self.store = torch.full((shift + rows * self.ld + 8,), 77.0, dtype=dtype, device=DEV) \
            if dtype.is_floating_point else torch.full((shift + rows * self.ld + 8,), 77, dtype=dtype, device=DEV)
        self.t = self.store[shift:].as_strided((rows, width), (self.ld, 1))
        if value is not None:
            self.t.copy_(value)

    @property
    def buf(self):
        z = self.store.element_size()
        return mm.Buf(self.store.data_ptr() + self.shift * z, ((self.rows - 1) * self.ld + self.width) * z)

    def cpu(self):
        torch.cuda.synchronize()
        return self.t.cpu()

    def untouched(self):
        """Everything outside the tensor still holds the sentinel."""
        probe = self.store.clone()
        probe[self.shift:].as_strided((self.rows, self.width), (self.ld, 1)).fill_(77)
        assert bool((probe == 77).all()), "written outside the output"


def u32(t):
    return t.numpy().view(np.uint32)


def ids_buf(ids: np.ndarray):
    return torch.from_numpy(ids.view(np.int32).copy()).to(DEV)


def f64(t):
    return t.double().numpy()


def near(got, want, bound, what):
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - want)[bad].max():.3e}"


# ---- router -------------------------------------------------------------------


def run_topk(logits, k, renormalize, ld=0, shift=0):
    m, E = logits.shape
    dt = {v: n for n, v in TORCH.items()}[logits.dtype]
    x = Padded(m, E, logits.dtype, ld, shift, logits)
    ids, w = Padded(m, k, torch.int32, 0, 1), Padded(m, k, torch.float32, 0, 1)
    p = mm.topk_params(dt, m, E, k, renormalize=renormalize, ld=ld)
    rec = mm.mm_topk(p, x.buf, ids.buf, w.buf, stream=stream())
    assert rec.kernel == mm.MM_KERNEL_TOPK and rec.route == mm.MM_ROUTE_TOPK and rec.dispatch_count == 1
    out = u32(ids.cpu()), f64(w.cpu())
    ids.untouched()
    w.untouched()
    return out


def check_topk(logits, k, renormalize, ld=0, shift=0):
    ids, w = run_topk(logits, k, renormalize, ld, shift)
    want_ids, want = ref.topk(f64(logits), k, renormalize)
    np.testing.assert_array_equal(ids, want_ids)
    # exp of an argument rounded at |l - peak| <= 128 that matters, its own two
    # steps, a sum of up to 22 levels, one division
    near(w, want, 160 * U * want + 1e-37, "weights")
    assert not np.signbit(w[want_ids == NONE]).any()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,E,k", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (5, 63, 7), (4, 65, 64), (7, 128, 1),
                                   (6, 200, 8), (9, 256, 8), (3, 511, 16), (2, 1000, 10), (2, 1024, 64), (130, 16, 2)])
@pytest.mark.parametrize("renormalize", [0, 1])
def test_topk(dt, m, E, k, renormalize):
    l = (torch.randn(m, E, generator=gen(m * E + k)) * 2).to(TORCH[dt])
    l[torch.rand(m, E, generator=gen(3)) < 0.1] = float("-inf")
    check_topk(l, k, renormalize)


@pytest.mark.parametrize("dt", DTYPES)
def test_topk_pitch_and_element_alignment(dt):
    l = torch.randn(6, 96, generator=gen(5)).to(TORCH[dt])
    check_topk(l, 8, 1, ld=101, shift=1)
    check_topk(l, 8, 0, ld=104, shift=0)


@pytest.mark.parametrize("E", [8, 96, 256])
def test_topk_equal_logits_go_to_the_lowest_expert(E):
    check_topk(torch.zeros(3, E), 8, 1)
    l = torch.randint(-2, 3, (40, E), generator=gen(7)).float()
    check_topk(l, 8, 0)
    l[:, ::2] = -0.0
    l[:, 1::2] = 0.0
    check_topk(l, 8, 0)  # both zeros are equal logits


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("renormalize", [0, 1])
def test_topk_masked_rows(dt, renormalize):
    low = torch.finfo(TORCH[dt]).min
    l = torch.randn(6, 70, generator=gen(9)).to(TORCH[dt])
    l[0] = float("-inf")              # nothing left
    l[1, 1:] = float("-inf")          # one left
    l[2] = low                        # the lowest value is a value, not a mask
    l[3, :68] = low
    l[4, 3:] = float("-inf")
    l[5, 0] = torch.finfo(TORCH[dt]).max
    check_topk(l, 4, renormalize)


@pytest.mark.parametrize("dt", [0, 2])
def test_topk_of_more_tokens_than_the_grid(dt):
    m, E, k = 65536 * (4 if dt == 0 else 16) + 77, 5, 2
    l = torch.randn(m, E, generator=gen(13)).to(TORCH[dt])
    ids, w = run_topk(l, k, 1)
    top = l.double().sort(dim=1, descending=True, stable=True)
    np.testing.assert_array_equal(ids, top.indices[:, :k].numpy().astype(np.uint32))
    want = torch.softmax(top.values[:, :k], 1).numpy()
    near(w, want, 160 * U * want, "weights")


@pytest.mark.parametrize("renormalize", [0, 1])
def test_topk_nan_and_inf(renormalize):
    l = torch.randn(4, 70, generator=gen(11))
    l[0, 5] = float("nan")
    l[1, :] = float("nan")
    l[2, 9] = float("inf")
    ids, w = run_topk(l, 3, renormalize)
    clean = l.clone()
    clean[0, 5] = float("-inf")
    want, _ = ref.topk(f64(clean), 3, renormalize)
    np.testing.assert_array_equal(ids[0], want[0])
    assert np.isnan(w[0]).all()
    assert (ids[1] == NONE).all() and (w[1] == 0).all()
    assert ids[2, 0] == 9 and np.isnan(w[2]).all()
    np.testing.assert_array_equal(ids[3], want[3])
    assert np.isfinite(w[3]).all()


@pytest.mark.parametrize("dt", [1, 2])
def test_topk_nan_and_inf_in_16_bits(dt):
    l = torch.randn(5, 70, generator=gen(12)).to(TORCH[dt])
    l[0, 5], l[0, 60] = float("nan"), -float("nan")
    l[1, :] = float("nan")
    l[2, 9] = float("inf")
    l[3, 1:] = float("-inf")
    for renormalize in (0, 1):
        ids, w = run_topk(l, 3, renormalize)
        clean = l.clone()
        clean[0, 5] = clean[0, 60] = float("-inf")
        want, _ = ref.topk(f64(clean), 3, renormalize)
        np.testing.assert_array_equal(ids[[0, 3, 4]], want[[0, 3, 4]])
        assert np.isnan(w[0]).all() and (ids[1] == NONE).all() and (w[1] == 0).all()
        assert ids[2, 0] == 9 and np.isnan(w[2]).all()
        assert w[3, 0] == 1 and (w[3, 1:] == 0).all() and np.isfinite(w[4]).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,E,k", [(1, 1, 1), (1, 64, 8), (5, 63, 7), (3, 65, 64), (6, 200, 8), (3, 511, 16),
                                   (2, 1024, 64), (33, 97, 6)])
@pytest.mark.parametrize("renormalize", [0, 1])
@pytest.mark.parametrize("pad", [0, 3])
def test_topk_grad(dt, m, E, k, renormalize, pad):
    l = (torch.randn(m, E, generator=gen(m + E)) * 1.5).to(TORCH[dt])
    l[torch.rand(m, E, generator=gen(4)) < 0.2] = float("-inf")
    if m > 2:
        l[1] = float("-inf")
    ids, _ = ref.topk(f64(l), k, renormalize)
    if m > 2:
        ids[2, 0] = E  # any id outside the experts is a slot without one
    g = torch.randn(m, k, generator=gen(6))
    gk = g.clone()
    gk[torch.from_numpy(ids >= E)] = float("nan")  # not used there
    x = Padded(m, E, TORCH[dt], E + pad, pad, l)
    d = Padded(m, E, TORCH[dt], E + pad, pad)
    di, dg = ids_buf(ids), gk.to(DEV)
    p = mm.topk_params(dt, m, E, k, renormalize=renormalize, ld=E + pad)
    rec = mm.mm_topk_grad(p, x.buf, mm.buf(di), mm.buf(dg), d.buf, stream=stream())
    assert rec.kernel == mm.MM_KERNEL_TOPK_GRAD
    want = ref.topk_grad(f64(l), ids, f64(g), bool(renormalize))
    # p to 160 steps as above, the dot product's 6 levels and g - dot
    scale = np.abs(f64(g)).max(1, keepdims=True)
    near(f64(d.cpu()), want, rounding(dt, want) + 400 * U * np.maximum(np.abs(want), 1e-2 * scale), "dlogits")
    d.untouched()


# ---- sorted rows --------------------------------------------------------------


def some_ids(m, k, E, seed, repeat=False, dropped=0.1):
    g = np.random.default_rng(seed)
    if repeat or k > E:
        ids = g.integers(0, E, size=(m, k))
    else:
        ids = np.stack([g.permutation(E)[:k] for _ in range(m)])
    ids = ids.astype(np.uint32)
    gone = g.random((m, k)) < dropped
    ids[gone] = g.choice(np.array([NONE, E, E + 7], dtype=np.uint32), size=int(gone.sum()))
    return ids


def run_sort(dt, x, ids, E, ld_t=0, ld_r=0, shift=0):
    m, h = x.shape
    k = ids.shape[1]
    R = m * k
    xt = Padded(m, h, TORCH[dt], ld_t, shift, x)
    xs = Padded(R, h, TORCH[dt], ld_r, shift)
    off, order, pos = (Padded(1, n, torch.int32, 0, 1) for n in (E + 1, R, R))
    di = ids_buf(ids)
    p = mm.sort_params(dt, m, k, E, h, ld_tokens=ld_t, ld_rows=ld_r)
    rec = mm.mm_id_sort(p, xt.buf, mm.buf(di), xs.buf, off.buf, order.buf, pos.buf, stream=stream())
    assert rec.route == mm.MM_ROUTE_SORT and rec.kernel == mm.MM_KERNEL_SORT_ROWS
    for b in (xs, off, order, pos):
        b.untouched()
    return xs, off, order, pos


SORT_SHAPES = [(1, 1, 1, 1), (1, 8, 64, 2048), (4, 8, 64, 513), (33, 6, 60, 96), (7, 2, 1000, 7), (3, 5, 2, 64),
               (100, 8, 1024, 17), (300, 4, 16, 40), (700, 7, 3, 33), (2100, 8, 129, 9)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,k,E,h", SORT_SHAPES)
def test_sort(dt, m, k, E, h):
    ids = some_ids(m, k, E, m + E, repeat=m % 2 == 0)
    x = torch.randn(m, h, generator=gen(m)).to(TORCH[dt])
    xs, off, order, pos = run_sort(dt, x, ids, E, *((h + 3, h + 5, 1) if h % 2 else (0, 0, 0)))
    w_off, w_order, w_pos = ref.plan(ids, E)
    np.testing.assert_array_equal(u32(off.cpu())[0], w_off)
    np.testing.assert_array_equal(u32(order.cpu())[0], w_order)
    np.testing.assert_array_equal(u32(pos.cpu())[0], w_pos)
    want = x[torch.from_numpy(w_order.astype(np.int64)) // k]
    want[int(w_off[E]):] = 0
    assert torch.equal(xs.cpu(), want)


@pytest.mark.parametrize("m,k,E", [(8200, 8, 40), (9000, 8, 5), (70001, 1, 300)])
def test_sort_plan_of_many_rows(m, k, E):
    """Up to and past the rows whose matches the plan keeps in registers (65536)."""
    ids = some_ids(m, k, E, E, repeat=True, dropped=0.05)
    x = torch.randn(m, 3, generator=gen(m))
    xs, off, order, pos = run_sort(0, x, ids, E)
    key = np.minimum(ids.reshape(-1).astype(np.int64), E)
    want = np.argsort(key, kind="stable")
    np.testing.assert_array_equal(u32(order.cpu())[0], want)
    np.testing.assert_array_equal(u32(off.cpu())[0], np.searchsorted(key[want], np.arange(E + 1)))
    place = np.empty(m * k, dtype=np.int64)
    place[want] = np.arange(m * k)
    np.testing.assert_array_equal(u32(pos.cpu())[0], place)
    rows = x[torch.from_numpy(want) // k]
    rows[int(u32(off.cpu())[0][E]):] = 0
    assert torch.equal(xs.cpu(), rows)


def test_sort_carries_bits():
    """NaN, infinities, denormals and -0 arrive as they are."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).reshape(64, 1024)
    x = bits.view(torch.float16)
    ids = some_ids(64, 2, 8, 1, dropped=0.0)
    xs, off, order, _ = run_sort(1, torch.zeros(64, 1024, dtype=torch.float16), ids, 8)
    xt, di = x.to(DEV), ids_buf(ids)
    out = torch.empty(128, 1024, dtype=torch.float16, device=DEV)
    p = mm.sort_params(1, 64, 2, 8, 1024)
    pos = torch.empty(128, dtype=torch.int32, device=DEV)
    mm.mm_id_sort(p, mm.buf(xt), mm.buf(di), mm.buf(out), off.buf, order.buf, mm.buf(pos), stream=stream())
    w_order = ref.plan(ids, 8)[1].astype(np.int64)
    assert torch.equal(out.cpu().view(torch.int16), bits[torch.from_numpy(w_order) // 2])


def test_sort_all_rows_without_an_expert():
    ids = np.full((9, 3), NONE, dtype=np.uint32)
    xs, off, order, pos = run_sort(2, torch.ones(9, 40).to(torch.bfloat16), ids, 12)
    assert (u32(off.cpu()) == 0).all() and (xs.cpu() == 0).all()
    np.testing.assert_array_equal(u32(order.cpu())[0], np.arange(27))
    np.testing.assert_array_equal(u32(pos.cpu())[0], np.arange(27))


def plan_dev(ids, E):
    off, order, pos = ref.plan(ids, E)
    return int(off[E]), pos, ids_buf(off), ids_buf(pos)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,k,E,h", SORT_SHAPES + [(3, 64, 64, 4100), (2, 3, 8, 9000)])
def test_sort_grad(dt, m, k, E, h):
    ids = some_ids(m, k, E, m + E + 1)
    if m > 2:
        ids[1] = NONE
    live, pos, doff, dpos = plan_dev(ids, E)
    dxs = torch.randn(m * k, h, generator=gen(m + 1)).to(TORCH[dt])
    dxs[live:] = float("nan")  # not read
    ld_t, ld_r, sh = (h + 3, h + 5, 1) if h % 2 else (0, 0, 0)
    src, out = Padded(m * k, h, TORCH[dt], ld_r, sh, dxs), Padded(m, h, TORCH[dt], ld_t, sh)
    p = mm.sort_params(dt, m, k, E, h, ld_tokens=ld_t, ld_rows=ld_r)
    mm.mm_id_sort_grad(p, src.buf, mm.buf(doff), mm.buf(dpos), out.buf, stream=stream())
    dxs[live:] = 0
    want, mag = ref.combine(f64(dxs), live, pos, np.ones((m, k)), None)
    near(f64(out.cpu()), want, rounding(dt, want) + (k + 1) * U * mag, "dx")
    out.untouched()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,k,E,h", SORT_SHAPES + [(3, 64, 64, 4100), (2, 3, 8, 9000)])
@pytest.mark.parametrize("residual", ["none", "apart", "in place"])
def test_combine(dt, m, k, E, h, residual):
    ids = some_ids(m, k, E, m + E + 2)
    if m > 2:
        ids[1] = NONE
    live, pos, doff, dpos = plan_dev(ids, E)
    y = torch.randn(m * k, h, generator=gen(m + 2)).to(TORCH[dt])
    y[live:] = float("nan")
    w = torch.rand(m, k, generator=gen(m + 3))
    wk = w.clone()
    wk[torch.from_numpy(ids >= E)] = float("inf")  # no slot, no weight
    res = torch.randn(m, h, generator=gen(m + 4)).to(TORCH[dt])
    ld_t, ld_r, sh = (h + 3, h + 5, 1) if h % 2 else (0, 0, 0)
    dy, out = Padded(m * k, h, TORCH[dt], ld_r, sh, y), Padded(m, h, TORCH[dt], ld_t, sh)
    dw = wk.to(DEV)
    rb = None
    if residual == "apart":
        keep = Padded(m, h, TORCH[dt], ld_t, sh, res)
        rb = keep.buf
    elif residual == "in place":
        out.t.copy_(res)
        rb = out.buf
    p = mm.sort_params(dt, m, k, E, h, ld_tokens=ld_t, ld_rows=ld_r)
    rec = mm.mm_id_combine(p, dy.buf, mm.buf(doff), mm.buf(dpos), mm.buf(dw), rb, out.buf, stream=stream())
    assert rec.kernel == mm.MM_KERNEL_COMBINE and rec.route == mm.MM_ROUTE_COMBINE
    y[live:] = 0
    want, mag = ref.combine(f64(y), live, pos, f64(w), None if residual == "none" else f64(res))
    near(f64(out.cpu()), want, rounding(dt, want) + (k + 1) * U * mag, "out")
    out.untouched()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,k,E,h", SORT_SHAPES + [(3, 64, 64, 4100), (2, 3, 8, 9000)])
def test_combine_grad(dt, m, k, E, h):
    ids = some_ids(m, k, E, m + E + 3)
    if m > 2:
        ids[1] = NONE
    live, pos, doff, dpos = plan_dev(ids, E)
    y = torch.randn(m * k, h, generator=gen(m + 5)).to(TORCH[dt])
    y[live:] = float("nan")
    d = torch.randn(m, h, generator=gen(m + 6)).to(TORCH[dt])
    w = torch.rand(m, k, generator=gen(m + 7))
    wk = w.clone()
    wk[torch.from_numpy(ids >= E)] = float("nan")
    ld_t, ld_r, sh = (h + 3, h + 5, 1) if h % 2 else (0, 0, 0)
    dd, dyin = Padded(m, h, TORCH[dt], ld_t, sh, d), Padded(m * k, h, TORCH[dt], ld_r, sh, y)
    dy, dw = Padded(m * k, h, TORCH[dt], ld_r, sh), Padded(m, k, torch.float32, 0, 1)
    dwt = wk.to(DEV)
    p = mm.sort_params(dt, m, k, E, h, ld_tokens=ld_t, ld_rows=ld_r)
    rec = mm.mm_id_combine_grad(p, dd.buf, dyin.buf, mm.buf(doff), mm.buf(dpos), mm.buf(dwt), dy.buf, dw.buf,
                                stream=stream())
    assert rec.kernel == mm.MM_KERNEL_COMBINE_GRAD
    y[live:] = 0
    want_dy, want_dw, mag = ref.combine_grad(f64(d), f64(y), live, pos, f64(w))
    near(f64(dy.cpu()), want_dy, rounding(dt, want_dy) + 2 * U * np.abs(want_dy), "dy")
    # a lane adds every 64th group of up to 8 elements, then 6 levels of the wave
    near(f64(dw.cpu()), want_dw, (h // 64 + 32) * U * mag, "dweights")
    dy.untouched()
    dw.untouched()


@pytest.mark.parametrize("dt", DTYPES)
def test_combine_of_rows_in_routed_order(dt):
    """Without position and offsets: rows as the expert-ID matmul leaves them."""
    m, k, E, h = 5, 3, 8, 70
    y = torch.randn(m * k, h, generator=gen(1)).to(TORCH[dt])
    w, d = torch.rand(m, k, generator=gen(2)), torch.randn(m, h, generator=gen(3)).to(TORCH[dt])
    out, dy, dw = Padded(m, h, TORCH[dt]), Padded(m * k, h, TORCH[dt]), Padded(m, k, torch.float32)
    yd, wd, dd = y.to(DEV), w.to(DEV), d.to(DEV)
    p = mm.sort_params(dt, m, k, E, h)
    mm.mm_id_combine(p, mm.buf(yd), None, None, mm.buf(wd), None, out.buf, stream=stream())
    mm.mm_id_combine_grad(p, mm.buf(dd), mm.buf(yd), None, None, mm.buf(wd), dy.buf, dw.buf, stream=stream())
    pos = np.arange(m * k)
    want, mag = ref.combine(f64(y), m * k, pos, f64(w), None)
    near(f64(out.cpu()), want, rounding(dt, want) + (k + 1) * U * mag, "out")
    want_dy, want_dw, mag = ref.combine_grad(f64(d), f64(y), m * k, pos, f64(w))
    near(f64(dy.cpu()), want_dy, rounding(dt, want_dy) + 2 * U * np.abs(want_dy), "dy")
    near(f64(dw.cpu()), want_dw, (h // 64 + 32) * U * mag, "dweights")


def test_sorted_rows_past_32_bit_offsets():
    """Rows 2^31 + 8 elements apart: byte and element offsets pass 32 bits."""
    m, k, E, h, ld = 2, 2, 4, 24, (1 << 31) + 8
    ids = np.array([[3, 1], [1, 0]], dtype=np.uint32)
    live, pos, doff, dpos = plan_dev(ids, E)
    rows = torch.empty(3 * ld + h, dtype=torch.bfloat16, device=DEV)
    view = rows.as_strided((4, h), (ld, 1))
    x = torch.randn(m, h, generator=gen(1)).to(torch.bfloat16)
    xd, w = x.to(DEV), torch.ones(m, k, device=DEV)
    off, order, p2 = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (E + 1, 4, 4))
    p = mm.sort_params(2, m, k, E, h, ld_rows=ld)
    mm.mm_id_sort(p, mm.buf(xd), mm.buf(ids_buf(ids)), mm.buf(rows), mm.buf(off), mm.buf(order), mm.buf(p2),
                  stream=stream())
    torch.cuda.synchronize()
    w_order = torch.from_numpy(ref.plan(ids, E)[1].astype(np.int64))
    assert torch.equal(view.cpu(), x[w_order // k])
    out = torch.empty(m, h, dtype=torch.bfloat16, device=DEV)
    mm.mm_id_combine(p, mm.buf(rows), mm.buf(doff), mm.buf(dpos), mm.buf(w), None, mm.buf(out), stream=stream())
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), (2 * x.float()).to(torch.bfloat16))


def test_bad_positions_stay_in_bounds():
    """Places past the rows are taken as slots without an expert."""
    m, k, E, h = 3, 2, 4, 24
    off = torch.tensor([0, 0, 0, 0, 1 << 30], dtype=torch.int32, device=DEV)
    pos = torch.tensor([0, 6, 1, 1 << 29, 2, -1], dtype=torch.int32, device=DEV)
    y, w = torch.ones(m * k, h, device=DEV), torch.ones(m, k, device=DEV)
    out, dy, dw = Padded(m, h, torch.float32), Padded(m * k, h, torch.float32), Padded(m, k, torch.float32)
    p = mm.sort_params(0, m, k, E, h)
    mm.mm_id_combine(p, mm.buf(y), mm.buf(off), mm.buf(pos), mm.buf(w), None, out.buf, stream=stream())
    mm.mm_id_combine_grad(p, out.buf, mm.buf(y), mm.buf(off), mm.buf(pos), mm.buf(w), dy.buf, dw.buf, stream=stream())
    assert (out.cpu() == 1).all()
    assert torch.equal(dw.cpu(), torch.tensor([[h, 0.0]] * 3))
    dy.untouched()


# ---- 4-bit products --------------------------------------------------------------


def q4_case(E, N, k, group, sdt, seed):
    g = gen(seed)
    codes = torch.randint(0, 256, (E, N, k // 2), generator=g, dtype=torch.int16).to(torch.uint8)
    scales = (torch.rand(E, N, k // group, generator=g) * 0.02 + 0.001).to(TORCH[sdt])
    biases = (torch.randn(E, N, k // group, generator=g) * 0.08).to(TORCH[sdt])
    return codes, scales, biases


def q4_dev(case):
    return tuple(t.to(DEV) for t in case)


def q4_check(y, dt, want, err, what):
    near(f64(y), want.numpy(), rounding(dt, want.numpy()) + err.numpy(), what)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("sdt", [1, 2])
@pytest.mark.parametrize("m,n,k,group", [
    (1, 1, 32, 32), (1, 16, 64, 64), (1, 33, 128, 128), (2, 17, 96, 32), (3, 40, 704, 64), (4, 100, 640, 128),
    (5, 31, 2080, 32), (7, 64, 4096, 64), (16, 19, 1408, 64), (17, 48, 384, 128), (37, 50, 1056, 32),
    (64, 130, 2048, 128), (1, 257, 8192, 32), (4, 16, 4224, 128)])
@pytest.mark.parametrize("gated", [0, 1])
def test_q4_gemv(dt, sdt, m, n, k, group, gated):
    case = q4_case(1, n * (1 + gated), k, group, sdt, n + k)
    x = torch.randn(m, k, generator=gen(k)).to(TORCH[dt])
    odd = n % 2
    xd = Padded(m, k, TORCH[dt], k + 3 * odd, odd, x)
    y = Padded(m, n, TORCH[dt], n + 5 * odd, odd)
    dev = q4_dev(case)
    p = mm.q4_params(dt, sdt, m, n, k, group, gated=gated, ldx=k + 3 * odd, ldy=n + 5 * odd)
    rec = mm.mm_q4_gemv(p, *(mm.buf(t) for t in dev), xd.buf, y.buf, stream=stream())
    assert rec.kernel == mm.MM_KERNEL_Q4 and rec.route == mm.MM_ROUTE_Q4
    want, err = ref.q4_product(case[0][0], case[1][0], case[2][0], group, x, bool(gated), dt == 0)
    q4_check(y.cpu(), dt, want, err, "y")
    y.untouched()


def routed(case, group, x_of_row, ids_of_row, gated, dt, n):
    R = len(ids_of_row)
    want, err = torch.zeros(R, n, dtype=torch.float64), torch.zeros(R, n, dtype=torch.float64)
    E = case[0].shape[0]
    for e in sorted(set(int(i) for i in ids_of_row)):
        if e >= E:
            continue
        at = torch.tensor([r for r in range(R) if int(ids_of_row[r]) == e])
        want[at], err[at] = ref.q4_product(case[0][e], case[1][e], case[2][e], group, x_of_row[at], gated, dt == 0)
    return want, err


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,k_slots,E,n,k,group", [(1, 8, 64, 70, 256, 32), (1, 1, 1, 16, 128, 128), (3, 2, 5, 33, 704, 64),
                                                   (9, 4, 6, 24, 2080, 32)])
@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("layout", [0, 1])
def test_q4_id_direct(dt, m, k_slots, E, n, k, group, gated, layout):
    case = q4_case(E, n * (1 + gated), k, group, 2, n + k)
    ids = some_ids(m, k_slots, E, m, repeat=True, dropped=0.2 if m > 1 else 0.0)
    R = m * k_slots
    x = torch.randn(m if layout == 0 else R, k, generator=gen(k)).to(TORCH[dt])
    y = Padded(R, n, TORCH[dt])
    dev, xd, di = q4_dev(case), x.to(DEV), ids_buf(ids)
    p = mm.q4_params(dt, 2, m, n, k, group, n_experts=E, top_k=k_slots, gated=gated, input_layout=layout)
    mm.mm_q4_id_direct(p, *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(di), y.buf, stream=stream())
    rows = x[torch.arange(R) // k_slots] if layout == 0 else x
    want, err = routed(case, group, rows, ids.reshape(-1), bool(gated), dt, n)
    q4_check(y.cpu(), dt, want, err, "y")
    none = torch.from_numpy(ids.reshape(-1) >= E)
    got = y.cpu()[none].float()
    assert (got == 0).all() and not torch.signbit(got).any()
    y.untouched()


def offsets_of(counts, R):
    off = np.zeros(len(counts) + 1, dtype=np.uint32)
    off[1:] = np.cumsum(counts)
    assert off[-1] <= R
    return off


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,k_slots,counts", [
    (1, 1, [1]), (1, 8, [1, 0, 3, 4]), (4, 5, [0, 17, 0, 0, 1]), (10, 8, [20, 1, 33, 0, 16, 4]),
    (8, 8, [0, 0, 0]), (50, 2, [100]), (3, 4, [1] * 5 + [0] * 600 + [2])])
@pytest.mark.parametrize("n,k,group,gated", [(24, 704, 64, 0), (33, 256, 32, 1), (17, 1152, 128, 0)])
def test_q4_id_sorted(dt, m, k_slots, counts, n, k, group, gated):
    E, R = len(counts), m * k_slots
    case = q4_case(E, n * (1 + gated), k, group, 1, n + k)
    off = offsets_of(counts, R)
    x = torch.randn(R, k, generator=gen(k)).to(TORCH[dt])
    x[int(off[-1]):] = float("nan")  # rows without an expert
    y = Padded(R, n, TORCH[dt], n + 3, 1)
    dev, xd, do = q4_dev(case), x.to(DEV), ids_buf(off)
    p = mm.q4_params(dt, 1, m, n, k, group, n_experts=E, top_k=k_slots, gated=gated, ldy=n + 3)
    mm.mm_q4_id_sorted(p, *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(do), y.buf, stream=stream())
    expert = np.full(R, NONE, dtype=np.uint32)
    for e in range(E):
        expert[off[e]:off[e + 1]] = e
    want, err = routed(case, group, x, expert, bool(gated), dt, n)
    q4_check(y.cpu(), dt, want, err, "y")
    y.untouched()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k,group,gated", [(61, 4100, 352, 32, 0), (50, 4201, 704, 64, 0), (11, 4100, 1152, 128, 1),
                                               (61, 16290, 352, 32, 0), (64, 16300, 704, 64, 0), (50, 8150, 640, 128, 1),
                                               (33, 8201, 1152, 128, 0)])
def test_q4_gemv_of_many_rows(dt, m, n, k, group, gated):
    """Enough blocks for two staged tiles a wave, and for waves that split the rows."""
    case = q4_case(1, n * (1 + gated), k, group, 1, n + k)
    x = torch.randn(m, k, generator=gen(k)).to(TORCH[dt])
    dev, xd, y = q4_dev(case), x.to(DEV), Padded(m, n, TORCH[dt])
    rec = mm.mm_q4_gemv(mm.q4_params(dt, 1, m, n, k, group, gated=gated), *(mm.buf(t) for t in dev), mm.buf(xd), y.buf,
                        stream=stream())
    if -(-m // 16) * -(-n // (64 if gated else 128)) >= 512:
        cols = 64 if gated else 128
    else:
        cols = 32 if dt != 0 and not gated and -(-m // 16) * -(-n // 16) >= 1024 else 16
    assert rec.variant == 16 + 256 * cols
    want, err = ref.q4_product(case[0][0], case[1][0], case[2][0], group, x, bool(gated), dt == 0)
    q4_check(y.cpu(), dt, want, err, "y")
    y.untouched()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("n,k,group,gated", [(800, 704, 64, 0), (333, 352, 32, 1), (801, 1152, 128, 0), (340, 256, 64, 1),
                                             (900, 32, 32, 0)])
def test_q4_id_sorted_of_many_rows(dt, n, k, group, gated):
    m, slots, E = 100, 8, 40
    R = m * slots
    counts = np.random.default_rng(n).multinomial(R - 30, np.random.default_rng(1).dirichlet(np.ones(E)))
    off = offsets_of(counts, R)
    case = q4_case(E, n * (1 + gated), k, group, 2, n + k)
    x = torch.randn(R, k, generator=gen(k)).to(TORCH[dt])
    x[int(off[-1]):] = float("nan")
    y = Padded(R, n, TORCH[dt], n + 1, 1)
    dev, xd, do = q4_dev(case), x.to(DEV), ids_buf(off)
    p = mm.q4_params(dt, 2, m, n, k, group, n_experts=E, top_k=slots, gated=gated, ldy=n + 1)
    rec = mm.mm_q4_id_sorted(p, *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(do), y.buf, stream=stream())
    assert rec.variant == 16 + 256 * (64 if gated else 128)
    expert = np.full(R, NONE, dtype=np.uint32)
    for e in range(E):
        expert[off[e]:off[e + 1]] = e
    want, err = routed(case, group, x, expert, bool(gated), dt, n)
    q4_check(y.cpu(), dt, want, err, "y")
    y.untouched()


def test_q4_more_tiles_than_one_grid_dimension():
    n, k, group = 3, 32, 32
    case = q4_case(1, n, k, group, 1, 5)
    dev = q4_dev(case)
    m = 16 * 33000 - 5
    x = torch.randn(m, k, generator=gen(1)).to(torch.float16)
    y, xd = Padded(m, n, torch.float16), x.to(DEV)
    mm.mm_q4_gemv(mm.q4_params(1, 1, m, n, k, group), *(mm.buf(t) for t in dev), mm.buf(xd), y.buf, stream=stream())
    want, err = ref.q4_product(case[0][0], case[1][0], case[2][0], group, x, False, False)
    q4_check(y.cpu(), 1, want, err, "y")
    m = 40000
    ids, y = torch.zeros(m, 1, dtype=torch.int32, device=DEV), Padded(m, n, torch.float16)
    mm.mm_q4_id_direct(mm.q4_params(1, 1, m, n, k, group), *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(ids), y.buf,
                       stream=stream())
    q4_check(y.cpu(), 1, want[:m], err[:m], "y by id")
    y.untouched()


def test_q4_sorted_offsets_that_lie_stay_in_bounds():
    m, ks, E, n, k = 5, 2, 4, 24, 128
    case = q4_dev(q4_case(E, n, k, 32, 1, 3))
    off = torch.tensor([0, 1 << 30, 3, -5, 2], dtype=torch.int32, device=DEV)
    x, y = torch.ones(m * ks, k, device=DEV), Padded(m * ks, n, torch.float32)
    p = mm.q4_params(0, 1, m, n, k, 32, n_experts=E, top_k=ks)
    mm.mm_q4_id_sorted(p, *(mm.buf(t) for t in case), mm.buf(x), mm.buf(off), y.buf, stream=stream())
    torch.cuda.synchronize()
    y.untouched()


def test_q4_other_rows_do_not_matter():
    """A row of NaN or infinities changes no other row."""
    case = q4_dev(q4_case(1, 40, 512, 32, 2, 1))
    for m in (3, 9):
        x = torch.randn(m, 512, generator=gen(2)).to(DEV)
        ys = []
        for bad in (0.0, float("nan"), float("inf")):
            z = x.clone()
            z[1] = bad
            y = torch.empty(m, 40, device=DEV)
            mm.mm_q4_gemv(mm.q4_params(0, 2, m, 40, 512, 32), *(mm.buf(t) for t in case), mm.buf(z), mm.buf(y),
                          stream=stream())
            torch.cuda.synchronize()
            ys.append(y.cpu())
        keep = [i for i in range(m) if i != 1]
        assert torch.equal(ys[0][keep], ys[1][keep]) and torch.equal(ys[0][keep], ys[2][keep])


def test_q4_codes_past_32_bit_offsets():
    """The last expert's codes lie past 4 GiB."""
    E, n, k, group = 37, 4096, 65536, 128
    codes = torch.empty(E, n, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.full((E, n, k // group), 0.01, dtype=torch.float16, device=DEV)
    biases = torch.full((E, n, k // group), -0.07, dtype=torch.float16, device=DEV)
    codes.zero_()
    last = torch.randint(0, 256, (n, k // 2), generator=gen(1), dtype=torch.int16).to(torch.uint8)
    codes[-1] = last.to(DEV)
    x = torch.randn(1, k, generator=gen(2)).to(torch.float16)
    y, xd = torch.empty(1, n, dtype=torch.float16, device=DEV), x.to(DEV)
    ids = ids_buf(np.array([[E - 1]], dtype=np.uint32))
    p = mm.q4_params(1, 1, 1, n, k, group, n_experts=E)
    mm.mm_q4_id_direct(p, mm.buf(codes), mm.buf(scales), mm.buf(biases), mm.buf(xd), mm.buf(ids), mm.buf(y),
                       stream=stream())
    torch.cuda.synchronize()
    rows = slice(n - 64, n)
    want, err = ref.q4_product(last[rows], scales[-1][rows], biases[-1][rows], group, x, False, False)
    q4_check(y[:, rows].cpu(), 1, want, err, "y")


# ---- streams, graphs -----------------------------------------------------------


def layer(dt=2, m=24, E=16, ks=4, h=256, n=96):
    g = gen(5)
    up, down = q4_dev(q4_case(E, 2 * n, h, 32, 2, 1)), q4_dev(q4_case(E, h, n, 32, 2, 2))
    t = TORCH[dt]
    R = m * ks
    b = dict(logits=torch.randn(m, E, generator=g).to(t).to(DEV), x=torch.randn(m, h, generator=g).to(t).to(DEV),
             ids=torch.empty(m, ks, dtype=torch.int32, device=DEV), w=torch.empty(m, ks, device=DEV),
             xs=torch.empty(R, h, dtype=t, device=DEV), off=torch.empty(E + 1, dtype=torch.int32, device=DEV),
             order=torch.empty(R, dtype=torch.int32, device=DEV), pos=torch.empty(R, dtype=torch.int32, device=DEV),
             mid=torch.empty(R, n, dtype=t, device=DEV), ys=torch.empty(R, h, dtype=t, device=DEV),
             out=torch.empty(m, h, dtype=t, device=DEV), dys=torch.empty(R, h, dtype=t, device=DEV),
             dw=torch.empty(m, ks, device=DEV), dl=torch.empty(m, E, dtype=t, device=DEV),
             dx=torch.empty(m, h, dtype=t, device=DEV))
    B = {k: mm.buf(v) for k, v in b.items()}
    pt, ps = mm.topk_params(dt, m, E, ks, renormalize=1), mm.sort_params(dt, m, ks, E, h)
    pu = mm.q4_params(dt, 2, m, n, h, 32, n_experts=E, top_k=ks, gated=1)
    pd = mm.q4_params(dt, 2, m, h, n, 32, n_experts=E, top_k=ks)

    def run(s):
        mm.mm_topk(pt, B["logits"], B["ids"], B["w"], stream=s)
        mm.mm_id_sort(ps, B["x"], B["ids"], B["xs"], B["off"], B["order"], B["pos"], stream=s)
        mm.mm_q4_id_sorted(pu, *(mm.buf(t) for t in up), B["xs"], B["off"], B["mid"], stream=s)
        mm.mm_q4_id_sorted(pd, *(mm.buf(t) for t in down), B["mid"], B["off"], B["ys"], stream=s)
        mm.mm_id_combine(ps, B["ys"], B["off"], B["pos"], B["w"], B["x"], B["out"], stream=s)
        mm.mm_id_combine_grad(ps, B["out"], B["ys"], B["off"], B["pos"], B["w"], B["dys"], B["dw"], stream=s)
        mm.mm_topk_grad(pt, B["logits"], B["ids"], B["dw"], B["dl"], stream=s)
        mm.mm_id_sort_grad(ps, B["dys"], B["off"], B["pos"], B["dx"], stream=s)

    outs = ("ids", "w", "xs", "off", "order", "pos", "mid", "ys", "out", "dys", "dw", "dl", "dx")
    return b, outs, run


def test_side_stream_and_graph_replays_give_the_eager_bits():
    b, outs, run = layer()
    side = torch.cuda.Stream()
    g = gen(8)
    run(stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(stream())
    for _ in range(4):
        b["logits"].copy_(torch.randn(b["logits"].shape, generator=g).to(b["logits"].dtype))
        b["x"].copy_(torch.randn(b["x"].shape, generator=g).to(b["x"].dtype))
        run(stream())
        torch.cuda.synchronize()
        eager = {n: b[n].clone() for n in outs}
        for n in outs:
            b[n].zero_()
        with torch.cuda.stream(side):
            run(side)
        side.synchronize()
        for n in outs:
            assert torch.equal(b[n], eager[n]), n
            b[n].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in outs:
            assert torch.equal(b[n], eager[n]), n
