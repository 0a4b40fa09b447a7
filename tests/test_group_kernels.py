"""The kernel that a grouped product takes follows from its sizes and type
(host only)."""
import ctypes
import os

import pytest

import bit_rank_post_amd as tq
from tests.group_cases import CASES, DW, DX, F8, IDS, Y, kernel_of, ragged


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(tq.LIB_PATH):
        pytest.skip("libtileq.so not built")


@pytest.mark.parametrize("product,kernel,groups,rows,d_in,d_out", CASES, ids=IDS)
def test_cases_take_the_kernel_they_are_meant_for(product, kernel, groups, rows, d_in, d_out):
    for act in (tq.TQ_F16, tq.TQ_BF16):
        assert kernel_of(product, groups, rows, d_in, d_out, act) == kernel
    counts = ragged(groups, rows, 2, 3)
    assert sum(counts) == rows - 5 and min(counts) >= 0 and len(counts) == groups


def test_every_kernel_has_a_case():
    rows = {(16, 16, 0), (32, 32, 0)}
    tiles = {(128, 32, 1), (128, 128, 1), (256, 256, 1)}
    want = {Y: rows | tiles, F8: rows | tiles, DX: tiles, DW: tiles - {(128, 32, 1)}}
    assert {p: {c[1] for c in CASES if c[0] == p} for p in want} == want
    # whatever the sizes, nothing else is taken
    for p in want:
        for g in (1, 3, 60, 64, 65, 1024):
            for r in (1, 17, 300, 5000, 70000, 1 << 20):
                for i in (16, 2048, 16384):
                    for o in (8, 1408, 16384):
                        assert kernel_of(p, g, r, i, o) in want[p]


def test_refusals():
    L, v = tq.lib(), [ctypes.byref(ctypes.c_int32()) for _ in range(3)]
    d = tq.GroupDesc(2, 64, 128, 64, tq.TQ_F16, 0x10000, None, 1, 64, 0, 0)
    b = ctypes.byref(d)
    assert L.tq_debug_group_kernel(b, 0, *v) == 0
    assert L.tq_debug_group_kernel(None, 0, *v) == 1
    assert L.tq_debug_group_kernel(b, 4, *v) == 1 and L.tq_debug_group_kernel(b, -1, *v) == 1
    for i in range(3):
        a = list(v)
        a[i] = None
        assert L.tq_debug_group_kernel(b, 0, *a) == 1
    d.d_in = 132
    assert L.tq_debug_group_kernel(b, 0, *v) == 2
