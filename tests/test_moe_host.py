"""Router, sorted rows and 4-bit products without a GPU: refusals (nothing is
enqueued) and the gradients' formulas against differences."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

import gemv_expert_id_amd as mm
import moe_ref as ref

BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(mm.LIB_PATH):
        from gemv_expert_id_amd import build
        build.build()
    return mm.load()


def _at(i, nbytes=BIG >> 4):
    """Fake device buffers far apart from each other (never dereferenced)."""
    return mm.Buf((i + 1) * BIG, nbytes)


def _fails(status, fn, *args):
    before = mm.load().mm_test_launch_count()
    with pytest.raises(mm.MmError) as ei:
        fn(*args)
    assert ei.value.status == status, str(ei.value)
    assert mm.load().mm_test_launch_count() == before, "enqueued despite the error"


INVALID, UNSUPPORTED, SMALL, MISALIGNED, OVERLAP = 1, 2, 3, 4, 5

# entry, params, exact bytes and element size of each buffer, names of the outputs' places
P_TOPK = mm.topk_params(2, 5, 12, 3)
P_SORT = mm.sort_params(2, 5, 3, 12, 40)
P_Q4 = mm.q4_params(0, 1, 5, 24, 64, 32)
P_Q4E = mm.q4_params(2, 2, 5, 24, 64, 32, n_experts=4, top_k=3, gated=1)
TOK, ROWS, SLOTS, OFF = 5 * 40 * 2, 15 * 40 * 2, 15 * 4, 13 * 4
CALLS = {
    "topk": (mm.mm_topk, P_TOPK, [(5 * 12 * 2, 2), (60, 4), (60, 4)], {1, 2}),
    "topk_grad": (mm.mm_topk_grad, P_TOPK, [(120, 2), (60, 4), (60, 4), (120, 2)], {3}),
    "sort": (mm.mm_id_sort, P_SORT, [(TOK, 2), (SLOTS, 4), (ROWS, 2), (OFF, 4), (SLOTS, 4), (SLOTS, 4)], {2, 3, 4, 5}),
    "sort_grad": (mm.mm_id_sort_grad, P_SORT, [(ROWS, 2), (OFF, 4), (SLOTS, 4), (TOK, 2)], {3}),
    "combine": (mm.mm_id_combine, P_SORT, [(ROWS, 2), (OFF, 4), (SLOTS, 4), (SLOTS, 4), (TOK, 2), (TOK, 2)], {5}),
    "combine_grad": (mm.mm_id_combine_grad, P_SORT,
                     [(TOK, 2), (ROWS, 2), (OFF, 4), (SLOTS, 4), (SLOTS, 4), (ROWS, 2), (SLOTS, 4)], {5, 6}),
    "q4_gemv": (mm.mm_q4_gemv, P_Q4, [(24 * 32, 16), (24 * 4, 2), (24 * 4, 2), (5 * 64 * 4, 4), (5 * 24 * 4, 4)], {4}),
    "q4_direct": (mm.mm_q4_id_direct, P_Q4E,
                  [(4 * 48 * 32, 16), (4 * 48 * 4, 2), (4 * 48 * 4, 2), (5 * 64 * 2, 2), (60, 4), (15 * 24 * 2, 2)], {5}),
    "q4_sorted": (mm.mm_q4_id_sorted, P_Q4E,
                  [(4 * 48 * 32, 16), (4 * 48 * 4, 2), (4 * 48 * 4, 2), (15 * 64 * 2, 2), (20, 4), (15 * 24 * 2, 2)], {5}),
}
INJECT = {"topk": "topk", "topk_grad": "topk_grad", "sort": "sort", "sort_grad": "sort", "combine": "combine",
          "combine_grad": "combine_grad", "q4_gemv": "q4", "q4_direct": "q4", "q4_sorted": "q4"}


def _copy(p, **kw):
    q = type(p).from_buffer_copy(p)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


@pytest.mark.parametrize("name", CALLS)
def test_exact_extents_are_enough_and_one_byte_less_is_not(name, lib):
    fn, p, bufs, _ = CALLS[name]
    exact = [_at(i, n) for i, (n, _) in enumerate(bufs)]
    lib.mm_test_inject_resolve_failure(INJECT[name].encode())
    _fails(UNSUPPORTED, fn, p, *exact)  # everything validated, then the injected failure
    for i in range(len(bufs)):
        short = list(exact)
        short[i] = mm.Buf(exact[i].ptr, bufs[i][0] - 1)
        _fails(SMALL, fn, p, *short)


@pytest.mark.parametrize("name", CALLS)
def test_null_and_misaligned_buffers(name):
    fn, p, bufs, _ = CALLS[name]
    for i, (_, align) in enumerate(bufs):
        args = [_at(j) for j in range(len(bufs))]
        args[i] = mm.Buf(args[i].ptr + align // 2, args[i].bytes)
        _fails(MISALIGNED, fn, p, *args)
        if name == "combine" and i == 4:
            continue  # the residual is optional
        args[i] = mm.Buf(None, 0)
        _fails(INVALID, fn, p, *args)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_overlap_nothing(name):
    fn, p, bufs, outs = CALLS[name]
    for o in outs:
        for i, (n, _) in enumerate(bufs):
            if i == o:
                continue
            args = [_at(j) for j in range(len(bufs))]
            args[o] = mm.Buf(args[i].ptr + (n - 1) // 16 * 16, args[o].bytes)  # meets its last bytes
            _fails(OVERLAP, fn, p, *args)


def test_combine_residual_in_place_or_apart(lib):
    fn, p, bufs, _ = CALLS["combine"]
    args = [_at(i, n) for i, (n, _) in enumerate(bufs)]
    args[4] = args[5]
    lib.mm_test_inject_resolve_failure(b"combine")
    _fails(UNSUPPORTED, fn, p, *args)
    args[4] = mm.Buf(args[5].ptr, args[5].bytes - 1)
    _fails(SMALL, fn, p, *args)
    args[4] = mm.Buf(args[5].ptr + 2, BIG >> 4)
    _fails(OVERLAP, fn, p, *args)


@pytest.mark.parametrize("name", ["combine", "combine_grad"])
def test_position_and_offsets_go_together(name, lib):
    fn, p, bufs, _ = CALLS[name]
    first = 1 if name == "combine" else 2
    args = [_at(i, n) for i, (n, _) in enumerate(bufs)]
    for i in (first, first + 1):
        some = list(args)
        some[i] = mm.Buf(None, 0)
        _fails(INVALID, fn, p, *some)
    args[first] = args[first + 1] = mm.Buf(None, 0)
    lib.mm_test_inject_resolve_failure(name.encode())
    _fails(UNSUPPORTED, fn, p, *args)


@pytest.mark.parametrize("name,field,value,status", [
    *[(n, "m", 0, INVALID) for n in CALLS],
    *[(n, "top_k", 0, INVALID) for n in CALLS],
    *[(n, "n_experts", 0, INVALID) for n in CALLS],
    *[(n, "dtype", 3, UNSUPPORTED) for n in CALLS],
    ("topk", "top_k", 13, INVALID), ("topk", "renormalize", 2, INVALID), ("topk", "reserved", 1, INVALID),
    ("topk", "n_experts", 1025, UNSUPPORTED), ("topk", "ld", 11, INVALID), ("topk", "ld", -1, INVALID),
    ("topk_grad", "ld", 1 << 62, INVALID),
    ("sort", "width", 0, INVALID), ("sort", "width", (1 << 24) + 1, INVALID), ("sort", "reserved", 1, INVALID),
    ("sort", "n_experts", 1025, UNSUPPORTED), ("sort", "m", 1 << 31, INVALID), ("sort", "ld_tokens", 39, INVALID),
    ("combine", "ld_rows", -40, INVALID), ("combine_grad", "ld_rows", 39, INVALID),
    ("sort_grad", "ld_rows", 1 << 61, INVALID),
    ("q4_gemv", "scale_dtype", 0, UNSUPPORTED), ("q4_gemv", "group", 16, UNSUPPORTED),
    ("q4_gemv", "group", 0, UNSUPPORTED), ("q4_gemv", "k", 96 + 16, INVALID), ("q4_gemv", "k", 0, INVALID),
    ("q4_gemv", "n", 0, INVALID), ("q4_gemv", "gated", 2, INVALID), ("q4_gemv", "n_experts", 2, INVALID),
    ("q4_gemv", "top_k", 2, INVALID), ("q4_gemv", "input_layout", 1, INVALID), ("q4_gemv", "ldx", 63, INVALID),
    ("q4_gemv", "ldy", 23, INVALID), ("q4_gemv", "ldx", 1 << 25, INVALID), ("q4_gemv", "k", 1 << 25, INVALID), ("q4_gemv", "n", (1 << 24) + 1, INVALID),
    ("q4_direct", "input_layout", 2, INVALID), ("q4_sorted", "input_layout", 1, INVALID),
    ("q4_sorted", "n_experts", 1025, UNSUPPORTED), ("q4_direct", "m", 1 << 31, INVALID),
])
def test_bad_fields(name, field, value, status):
    fn, p, bufs, _ = CALLS[name]
    _fails(status, fn, _copy(p, **{field: value}), *[_at(i) for i in range(len(bufs))])


def test_topk_slots_limit():
    _fails(UNSUPPORTED, mm.mm_topk, mm.topk_params(0, 2, 100, 65), _at(0), _at(1), _at(2))


@pytest.mark.parametrize("name", CALLS)
def test_null_params(name, lib):
    _, _, bufs, _ = CALLS[name]
    args = [_at(i) for i in range(len(bufs))]
    entry = getattr(lib, CALLS[name][0].__name__)
    assert entry(None, *args, ctypes.c_void_p(0), None) == INVALID


def test_plan_of_no_experts_and_repeats():
    off, order, pos = ref.plan(np.array([[2, 2], [ref.NONE, 0]], dtype=np.uint32), 3)
    assert off.tolist() == [0, 1, 1, 3] and order.tolist() == [3, 0, 1, 2] and pos.tolist() == [1, 2, 3, 0]


@pytest.mark.parametrize("renormalize", [False, True])
def test_topk_gradient_formula_against_differences(renormalize):
    rng = np.random.default_rng(1)
    l = rng.normal(size=(3, 9))
    l[1, 4] = -np.inf
    l[2, 2:] = -np.inf
    ids, _ = ref.topk(l, 4, renormalize)
    g = rng.normal(size=ids.shape)
    got = ref.topk_grad(l, ids, g, renormalize)
    h = 1e-6
    for t in range(3):
        for e in range(9):
            if l[t, e] == -np.inf:
                assert got[t, e] == 0
                continue
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            iu, wu = ref.topk(up, 4, renormalize)
            idn, wd = ref.topk(down, 4, renormalize)
            assert (iu == ids).all() and (idn == ids).all()
            live = ids[t] < 9
            diff = ((wu - wd)[t, live] * g[t, live]).sum() / (2 * h)
            assert abs(diff - got[t, e]) < 1e-8


def test_combine_gradient_formula_against_differences():
    rng = np.random.default_rng(2)
    m, k, E, h = 4, 2, 3, 5
    ids = rng.integers(0, E, size=(m, k)).astype(np.uint32)
    ids[1, 1] = ref.NONE
    off, _, pos = ref.plan(ids, E)
    y, w, d = rng.normal(size=(m * k, h)), rng.normal(size=(m, k)), rng.normal(size=(m, h))
    dy, dw, _ = ref.combine_grad(d, y, int(off[E]), pos, w)
    f = lambda y, w: (ref.combine(y, int(off[E]), pos, w, None)[0] * d).sum()  # noqa: E731
    step = 1e-5
    for arr, grad, at in ((y, dy, 0), (w, dw, 1)):
        for idx in np.ndindex(arr.shape):
            up, down = arr.copy(), arr.copy()
            up[idx] += step
            down[idx] -= step
            diff = (f(up, w) - f(down, w) if at == 0 else f(y, up) - f(y, down)) / (2 * step)
            assert abs(diff - grad[idx]) < 1e-8
