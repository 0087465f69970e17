"""Feed-forward block without a GPU: refusals (nothing is enqueued) and the
gradient's formula against differences."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import ffn_ref as ref
import gemv_expert_id_amd as mm

BIG = 1 << 42


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

# entry, params, exact bytes and alignment of each buffer, places of outputs, places that may be absent
X, W, PRE, H = 5 * 40 * 2, 48 * 40 * 2, 5 * 48 * 2, 5 * 24 * 2
P_GATED = mm.gated_params(2, 5, 24, 40)
CALLS = {
    "gated": (mm.mm_gated, P_GATED, [(X, 2), (W, 2), (H, 2), (PRE, 2)], {2, 3}, {3}),
    "gated_grad": (mm.mm_gated_grad, P_GATED, [(X, 2), (W, 2), (PRE, 2), (H, 2), (PRE, 2), (X, 2), (W, 2)], {4, 5, 6},
                   {2, 5, 6}),
    "quant": (mm.mm_i8_quant, mm.quant_params(0, 5, 33), [(5 * 33 * 4, 4), (5 * 33, 1), (20, 4)], {1, 2}, set()),
    "i8": (mm.mm_i8_gemm, mm.i8_params(1, 5, 24, 48), [(5 * 48, 16), (20, 4), (24 * 48, 16), (96, 4), (5 * 24 * 2, 2)],
           {4}, set()),
    "i8_gated": (mm.mm_i8_gemm, mm.i8_params(0, 5, 24, 48, gate=1),
                 [(5 * 48, 16), (20, 4), (48 * 48, 16), (192, 4), (5 * 24 * 4, 4)], {4}, set()),
}
INJECT = {"gated": "gated", "gated_grad": "gated_grad", "quant": "i8_quant", "i8": "i8", "i8_gated": "i8"}


def _copy(p, **kw):
    q = type(p).from_buffer_copy(p)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


@pytest.mark.parametrize("name", CALLS)
def test_exact_extents_are_enough_and_one_byte_less_is_not(name, lib):
    fn, p, bufs, _, _ = CALLS[name]
    exact = [_at(i, n) for i, (n, _) in enumerate(bufs)]
    lib.mm_test_inject_resolve_failure(INJECT[name].encode())
    _fails(UNSUPPORTED, fn, p, *exact)  # everything validated, then the injected failure
    for i in range(len(bufs)):
        short = list(exact)
        short[i] = mm.Buf(exact[i].ptr, bufs[i][0] - 1)
        _fails(SMALL, fn, p, *short)


@pytest.mark.parametrize("name", CALLS)
def test_extents_with_pitches(name, lib):
    """Rows a pitch apart, the last one as long as its row."""
    fn, p, bufs, _, _ = CALLS[name]
    es = 4 if p.dtype == 0 else 2
    if name.startswith("gated"):
        p = _copy(p, ldx=41, ldw=50, ldpre=49, ldh=31)
        z = {X: 4 * 41 * 2 + 80, W: 47 * 50 * 2 + 80, PRE: 4 * 49 * 2 + 96, H: 4 * 31 * 2 + 48}
        need = [z[n] for n, _ in bufs]
    elif name == "quant":
        p = _copy(p, ldx=35, ldq=34)
        need = [(4 * 35 + 33) * 4, 4 * 34 + 33, 20]
    else:
        p = _copy(p, ldx=64, ldw=80, ldy=25)
        rows = 24 * (1 + (p.gate > 0))
        need = [4 * 64 + 48, 20, (rows - 1) * 80 + 48, rows * 4, (4 * 25 + 24) * es]
    exact = [_at(i, n) for i, n in enumerate(need)]
    lib.mm_test_inject_resolve_failure(INJECT[name].encode())
    _fails(UNSUPPORTED, fn, p, *exact)
    for i in range(len(need)):
        short = list(exact)
        short[i] = mm.Buf(exact[i].ptr, need[i] - 1)
        _fails(SMALL, fn, p, *short)


@pytest.mark.parametrize("name", CALLS)
def test_null_and_misaligned_buffers(name, lib):
    fn, p, bufs, _, optional = CALLS[name]
    for i, (_, align) in enumerate(bufs):
        args = [_at(j) for j in range(len(bufs))]
        if align > 1:
            args[i] = mm.Buf(args[i].ptr + align // 2, args[i].bytes)
            _fails(MISALIGNED, fn, p, *args)
        args[i] = mm.Buf(None, 0)
        if i in optional:
            lib.mm_test_inject_resolve_failure(INJECT[name].encode())
            _fails(UNSUPPORTED, fn, p, *args)
        else:
            _fails(INVALID, fn, p, *args)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_overlap_nothing(name):
    fn, p, bufs, outs, _ = CALLS[name]
    for o in outs:
        for i, (n, _) in enumerate(bufs):
            if i == o:
                continue
            args = [_at(j) for j in range(len(bufs))]
            args[o] = mm.Buf(args[i].ptr + (n - 1) // 16 * 16, args[o].bytes)  # meets its last bytes
            _fails(OVERLAP, fn, p, *args)


def test_gradient_in_place_of_the_pre_activations(lib):
    fn, p, bufs, _, _ = CALLS["gated_grad"]
    args = [_at(i, n) for i, (n, _) in enumerate(bufs)]
    args[2] = args[4]
    lib.mm_test_inject_resolve_failure(b"gated_grad")
    _fails(UNSUPPORTED, fn, p, *args)
    args[2] = mm.Buf(args[4].ptr, args[4].bytes - 1)
    _fails(SMALL, fn, p, *args)
    args[2] = mm.Buf(args[4].ptr + 2, BIG >> 4)
    _fails(OVERLAP, fn, p, *args)


@pytest.mark.parametrize("name,field,value,status", [
    *[(n, f, 0, INVALID) for n in CALLS for f in ("m", "k")],
    *[(n, "n", 0, INVALID) for n in CALLS if n != "quant"],
    *[(n, "dtype", 3, UNSUPPORTED) for n in CALLS],
    *[(n, "reserved", 1, INVALID) for n in CALLS],
    *[(n, "m", 1 << 31, INVALID) for n in CALLS],
    *[(n, "m", (1 << 24) + 1, INVALID) for n in CALLS if n != "quant"],
    *[(n, "n", (1 << 24) + 1, INVALID) for n in CALLS if n != "quant"],
    *[(n, "ldx", v, INVALID) for n in CALLS for v in (-48, 1, 1 << 62)],
    ("gated", "gate", 0, INVALID), ("gated", "gate", 3, INVALID), ("gated_grad", "gate", 0, INVALID),
    ("i8", "gate", 3, INVALID), ("gated", "k", (1 << 24) + 1, INVALID), ("quant", "k", (1 << 24) + 1, INVALID),
    ("gated", "ldw", 39, INVALID), ("gated", "ldpre", 47, INVALID), ("gated_grad", "ldh", 23, INVALID),
    ("quant", "ldq", 32, INVALID), ("i8", "ldw", 47, INVALID), ("i8", "ldy", 23, INVALID),
    ("i8", "k", 40, INVALID), ("i8", "k", 131072, INVALID), ("i8", "ldx", 56, INVALID), ("i8", "ldw", 1 << 24, INVALID),
])
def test_bad_fields(name, field, value, status):
    fn, p, bufs, _, _ = CALLS[name]
    _fails(status, fn, _copy(p, **{field: value}), *[_at(i) for i in range(len(bufs))])


@pytest.mark.parametrize("name", [n for n in CALLS if n != "quant"])
def test_largest_outputs(name):
    fn, p, bufs, _, _ = CALLS[name]
    _fails(INVALID, fn, _copy(p, m=(1 << 18) + 1, n=1 << 18), *[_at(i, BIG) for i in range(len(bufs))])


@pytest.mark.parametrize("name", CALLS)
def test_null_params(name, lib):
    _, _, bufs, _, _ = CALLS[name]
    args = [_at(i) for i in range(len(bufs))]
    entry = getattr(lib, CALLS[name][0].__name__)
    assert entry(None, *args, ctypes.c_void_p(0), None) == INVALID


@pytest.mark.parametrize("gate", [ref.SILU, ref.GELU])
def test_gradient_formula_against_differences(gate):
    g = torch.Generator().manual_seed(3)
    x, w, dh = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 5), (8, 5), (3, 4)))
    f = lambda x, w: float((ref.gated(x, w, gate)[0] * dh).sum())  # noqa: E731
    _, pre, _, e = ref.gated(x, w, gate)
    dpre, _ = ref.gated_grad(pre, e, dh, gate)
    step = 1e-5
    for t, grad in ((x, dpre @ w), (w, dpre.t() @ x)):
        for i in range(t.numel()):
            up, down = t.clone(), t.clone()
            up.view(-1)[i] += step
            down.view(-1)[i] -= step
            diff = (f(up, w) - f(down, w) if t is x else f(x, up) - f(x, down)) / (2 * step)
            assert abs(diff - float(grad.reshape(-1)[i])) < 1e-7


@pytest.mark.parametrize("gate", [ref.SILU, ref.GELU])
def test_slope_and_curvature_bounds(gate):
    a = torch.linspace(-20, 20, 400001, dtype=torch.float64)
    s = ref.act_slope(a, gate)
    assert float(s.abs().max()) < ref.SLOPE
    assert float((s.diff() / a.diff()).abs().max()) < ref.CURVE


def test_codes_of_borders_and_zero_rows():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, 63.5], [0.0, 0, 0, 0, 0], [2.0 ** -125, 2.0 ** -126, 2.0 ** -127, 0, 0]])
    q, s = ref.quantise(x)
    assert q.tolist() == [[127, 0, 2, -2, 64], [0] * 5, [2, 1, 0, 0, 0]]
    assert s.tolist() == [1.0, 2.0 ** -126, 2.0 ** -126]
