"""The rule for the launches of mm_id_sort, compiled for the host: what the one
launch reads is bounded for every accepted size."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemv_expert_id_amd", "csrc")


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text('#include "sort_rule.hpp"\n'
                                'extern "C" int launches(unsigned m, unsigned k) { return mmk::sort_launches(m, k); }\n')
    lib = str(d / "rule.so")
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "rule.cpp"), "-o", lib], check=True)
    fn = ctypes.CDLL(lib).launches
    fn.argtypes = [ctypes.c_uint, ctypes.c_uint]
    return fn


def test_ids_that_the_one_launch_reads_are_bounded(launches):
    """Each of m blocks reads m * top_k ids once for each eight slots, one round after the other."""
    sizes = sorted({v for i in range(31) for v in ((1 << i) - 1, 1 << i, (1 << i) + 1, 3 << i) if 0 < v < 1 << 31})
    for m in sizes:
        for k in sizes:
            if m * k >= 1 << 31:
                continue
            rounds = -(-k // 8)
            if launches(m, k) == 1:
                assert m * m * k * rounds <= 1 << 21 and rounds <= 2, (m, k)
            else:
                assert m * m * k * rounds > 1 << 21 or rounds > 2, (m, k)


@pytest.mark.parametrize("m,k,want", [
    (1, 1, 1), (4, 8, 1), (512, 8, 1), (513, 8, 2), (256, 16, 1), (362, 16, 2), (1448, 1, 1), (1449, 1, 2),
    (1, 16, 1), (1, 17, 2), (1, 64, 2), (181, 64, 2), (1, 1024, 2), (8, 32768, 2), (1, 1 << 21, 2),
    (1, (1 << 31) - 1, 2), ((1 << 31) - 1, 1, 2), (46340, 46340, 2)])
def test_launches_at_given_sizes(launches, m, k, want):
    assert launches(m, k) == want
