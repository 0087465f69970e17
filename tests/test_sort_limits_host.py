"""Slots per token of the sorted-row calls: a token's rows are added one after
the other, so their number is limited."""
from __future__ import annotations

import os

import pytest

import gemv_expert_id_amd as mm

FAR = 1 << 44
ROWS = (1 << 31) - 1
# entry and number of its buffers
CALLS = {"sort": (mm.mm_id_sort, 6), "sort_grad": (mm.mm_id_sort_grad, 4), "combine": (mm.mm_id_combine, 6),
         "combine_grad": (mm.mm_id_combine_grad, 7)}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(mm.LIB_PATH):
        from gemv_expert_id_amd import build
        build.build()
    return mm.load()


def refused(name, top_k):
    fn, n = CALLS[name]
    before = mm.load().mm_test_launch_count()
    bufs = [mm.Buf((i + 1) * FAR, FAR >> 1) for i in range(n)]
    with pytest.raises(mm.MmError) as e:
        fn(mm.sort_params(0, 1, top_k, 4, 1), *bufs)
    assert e.value.status == 2 and mm.load().mm_test_launch_count() == before
    return str(e.value)


@pytest.mark.parametrize("name", CALLS)
def test_slots_are_limited(name, lib):
    for k in (mm.MM_SORT_MAX_SLOTS + 1, 1 << 21, ROWS):
        assert "slots" in refused(name, k)
    # the largest is taken: only the injected failure stops it
    lib.mm_test_inject_resolve_failure({"sort_grad": b"sort"}.get(name, name.encode()))
    assert "injected" in refused(name, mm.MM_SORT_MAX_SLOTS)
