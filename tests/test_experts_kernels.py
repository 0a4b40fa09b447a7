"""The kernels of the layer for a few tokens follow from the sizes, and the cases
that the GPU tests run take all of them (host only)."""
import ctypes

import pytest

import bit_rank_post_amd as tq
from tests.experts_cases import CASES8, CASES16, kernels_of
from tests.test_abi_layer_ops import L, refused  # noqa: F401  (L: fixture)


@pytest.mark.parametrize("int8,cases", [(0, CASES16), (1, CASES8)])
def test_cases_take_all_kernels(L, int8, cases):  # noqa: F811
    for columns, up, down, E, T, k, d, ff, hot in cases:
        assert kernels_of(T, k, E, d, ff, int8) == (columns, up, down), (E, T, k, d, ff)
        assert hot <= T * k
    kinds = {c[:3] for c in cases}
    step = 16 if int8 else 8
    for E in (1, 2, 8, 60, 64, 256, 1024):
        for T in (1, 2, 16, 17, 32, 33, 128, 1024):
            for k in (1, 2, 8):
                for d in (step, 256, 2048, 4000, 4096, 8192, 65536):
                    for ff in (step, 256, 2048, 4096, 8192, 65536):
                        if T * k <= 1024:
                            assert kernels_of(T, k, E, d, ff, int8) in kinds, (E, T, k, d, ff)


def test_refusals(L):  # noqa: F811
    c, up, down = ctypes.byref(ctypes.c_int32()), (ctypes.c_int32 * 2)(), (ctypes.c_int32 * 2)()
    f = L.tq_debug_experts_kernels
    for args in ((None, up, down), (c, None, down), (c, up, None)):
        refused(L, f(4, 2, 8, 64, 32, 0, *args), 1, b"NULL")
    for sizes, code in (((0, 2, 8, 64, 32, 0), 2), ((-1, 2, 8, 64, 32, 0), 2), ((4, 0, 8, 64, 32, 0), 2), ((4, 2, 0, 64, 32, 0), 2),
                        ((4, 2, 8, 60, 32, 0), 2), ((4, 2, 8, 64, 40, 1), 2), ((513, 2, 8, 64, 32, 0), 5)):
        assert f(*sizes, c, up, down) == code
    assert "tq_debug_experts_kernels" in tq.EXPORTS
