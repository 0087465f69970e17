"""Rows without an expert behind the sorted ones of mm_q4_id_sorted: written as
zeros whatever their number, in every form, and at no more than the time that
the same rows take with an expert."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemv_expert_id_amd as mm
from test_gpu_moe import DTYPES, Padded, TORCH, gen, ids_buf, offsets_of, q4_case, q4_check, q4_dev, routed, stream, NONE

pytestmark = pytest.mark.gpu


# rows with an expert in each of four experts, of 700 rows; outputs that lead to
# 4 tokens a tile, 16 with k split, with two tiles a wave, and waves that share x
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts", [[0, 0, 0, 0], [1, 0, 0, 0], [0, 16, 3, 0], [100, 0, 17, 233], [0, 0, 0, 699]])
@pytest.mark.parametrize("n", [33, 700, 2500])
@pytest.mark.parametrize("gated", [0, 1])
def test_rows_without_an_expert_are_zeros(dt, counts, n, gated):
    E, R, k, group = 4, 700, 96, 32
    case = q4_case(E, n * (1 + gated), k, group, 1, n)
    off = offsets_of(counts, R)
    x = torch.randn(R, k, generator=gen(n)).to(TORCH[dt])
    x[int(off[-1]):] = float("nan")
    y = Padded(R, n, TORCH[dt], n + 3, 1)
    dev, xd, do = q4_dev(case), x.to("cuda:0"), ids_buf(off)
    p = mm.q4_params(dt, 1, R, n, k, group, n_experts=E, top_k=1, gated=gated, ldy=n + 3)
    mm.mm_q4_id_sorted(p, *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(do), y.buf, stream=stream())
    expert = np.full(R, NONE, dtype=np.uint32)
    for e in range(E):
        expert[off[e]:off[e + 1]] = e
    want, err = routed(case, group, x, expert, bool(gated), dt, n)
    got = y.cpu()
    q4_check(got, dt, want, err, "y")
    assert not torch.signbit(got[int(off[-1]):].float()).any()
    y.untouched()


def test_rows_without_an_expert_of_few_rows():
    """Tiles of 4 tokens: at most 4 rows an expert."""
    E, R, n, k = 40, 130, 50, 64
    case = q4_case(E, n, k, 64, 2, 1)
    for live in (0, 1, 5, 128, 130):
        counts = np.bincount(np.arange(live) * 7 % E, minlength=E)
        off = offsets_of(counts, R)
        x = torch.randn(R, k, generator=gen(live)).to(torch.bfloat16)
        x[live:] = float("nan")
        y = Padded(R, n, torch.bfloat16)
        dev, xd, do = q4_dev(case), x.to("cuda:0"), ids_buf(off)
        p = mm.q4_params(2, 2, R, n, k, 64, n_experts=E, top_k=1)
        rec = mm.mm_q4_id_sorted(p, *(mm.buf(t) for t in dev), mm.buf(xd), mm.buf(do), y.buf, stream=stream())
        assert rec.variant == 4 + 256 * 16
        expert = np.full(R, NONE, dtype=np.uint32)
        for e in range(E):
            expert[off[e]:off[e + 1]] = e
        want, err = routed(case, 64, x, expert, False, 2, n)
        q4_check(y.cpu(), 2, want, err, "y")
        y.untouched()


@pytest.mark.parametrize("share", [0.5, 1.0])
def test_rows_without_an_expert_take_no_longer(share):
    """65536 routed rows, `share` of them without an expert. Their zeros are fewer
    bytes than the products' operands, so the call may take no longer; half as
    long again is allowed for timing."""
    E, R, n, k = 64, 65536, 256, 256
    dev = q4_dev(q4_case(E, n, k, 64, 2, 1))
    x, y = torch.randn(R, k, generator=gen(1)).to(torch.bfloat16).to("cuda:0"), Padded(R, n, torch.bfloat16)
    p = mm.q4_params(2, 2, R, n, k, 64, n_experts=E, top_k=1)
    best = {}
    for gone in (0.0, share):
        off = ids_buf(offsets_of([int(R * (1 - gone)) // E] * E, R))
        times = []
        for _ in range(10):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            mm.mm_q4_id_sorted(p, *(mm.buf(t) for t in dev), mm.buf(x), mm.buf(off), y.buf, stream=stream())
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        best[gone] = min(times)
    print({g: f"{1000 * t:.1f} us" for g, t in best.items()})
    assert best[share] <= 1.5 * best[0.0], best
