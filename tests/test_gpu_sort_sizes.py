"""The sort past the sizes of test_gpu_moe.py: many slots a token, rows of
several pieces, and its two launches in a graph."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemv_expert_id_amd as mm
import moe_ref as ref
from test_gpu_moe import DEV, DTYPES, TORCH, gen, ids_buf, run_sort, some_ids, stream, u32

pytestmark = pytest.mark.gpu


def expect_sort(x, ids, E, xs, off, order, pos):
    m, k = ids.shape
    key = np.minimum(ids.reshape(-1).astype(np.int64), E)
    w_order = np.argsort(key, kind="stable")
    w_off = np.searchsorted(key[w_order], np.arange(E + 1))
    w_pos = np.empty(m * k, dtype=np.int64)
    w_pos[w_order] = np.arange(m * k)
    np.testing.assert_array_equal(u32(off.cpu())[0], w_off)
    np.testing.assert_array_equal(u32(order.cpu())[0], w_order)
    np.testing.assert_array_equal(u32(pos.cpu())[0], w_pos)
    want = x[torch.from_numpy(w_order) // k]
    want[int(w_off[E]):] = 0
    assert torch.equal(xs.cpu(), want)


@pytest.mark.parametrize("m,k,E,h", [
    (1, 9, 16, 40), (1, 16, 64, 513), (2, 17, 8, 96), (5, 24, 300, 33), (9, 64, 64, 65), (40, 33, 1024, 24),
    (1, 65, 70, 40), (2, 200, 3, 33), (1, 1024, 1024, 16), (8, 300, 5, 17), (3, 2049, 60, 9)])
@pytest.mark.parametrize("dt", DTYPES)
def test_sort_of_many_slots(dt, m, k, E, h):
    ids = some_ids(m, k, E, m + k, repeat=k % 2 == 1)
    x = torch.randn(m, h, generator=gen(m)).to(TORCH[dt])
    expect_sort(x, ids, E, *run_sort(dt, x, ids, E, *((h + 3, h + 5, 1) if h % 2 else (0, 0, 0))))


@pytest.mark.parametrize("m,k,E,h", [(1, 8, 16, 4097), (4, 2, 5, 8192), (3, 11, 64, 12300), (33, 8, 60, 9001),
                                     (400, 8, 8, 8192), (600, 9, 200, 4101), (1100, 3, 7, 8196)])
@pytest.mark.parametrize("dt", [0, 2])
def test_sort_of_rows_of_several_pieces(dt, m, k, E, h):
    ids = some_ids(m, k, E, h, repeat=False)
    x = torch.randn(m, h, generator=gen(m)).to(TORCH[dt])
    expect_sort(x, ids, E, *run_sort(dt, x, ids, E, *((h + 3, h + 5, 1) if h % 2 else (0, 0, 0))))


def test_two_launches_of_the_sort_in_a_graph():
    """m * m * top_k above 2^21: a plan, then the rows; replayed with new ids and rows each time."""
    m, k, E, h = 2100, 3, 24, 40
    R = m * k
    x = torch.empty(m, h, dtype=torch.bfloat16, device=DEV)
    ids = torch.empty(m, k, dtype=torch.int32, device=DEV)
    outs = [torch.empty(R, h, dtype=torch.bfloat16, device=DEV)] + [
        torch.empty(n, dtype=torch.int32, device=DEV) for n in (E + 1, R, R)]
    p = mm.sort_params(2, m, k, E, h)

    def run():
        return mm.mm_id_sort(p, mm.buf(x), mm.buf(ids), *(mm.buf(o) for o in outs), stream=stream())

    def fill(seed):
        x.copy_(torch.randn(m, h, generator=gen(seed)))
        ids.copy_(torch.from_numpy(some_ids(m, k, E, seed).view(np.int32)))

    fill(0)
    assert run().dispatch_count == 2
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(1, 5):
        fill(seed)
        run()
        torch.cuda.synchronize()
        eager = [o.clone() for o in outs]
        w_off, w_order, _ = ref.plan(some_ids(m, k, E, seed), E)
        np.testing.assert_array_equal(u32(outs[1].cpu()), w_off)
        np.testing.assert_array_equal(u32(outs[2].cpu()), w_order)
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e)
