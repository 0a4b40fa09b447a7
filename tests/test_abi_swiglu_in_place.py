"""Outputs of SwiGLU and its gradient that start in a half of a's or da's rows
with another type or row stride are refused (host only): rows would be written
where others, not yet read, lie, or two outputs in one place."""
import ctypes

import pytest

from tests.test_abi_layer_ops import L, P, Q, R, refused, swiglu  # noqa: F401  (L: fixture)

FF = 64


@pytest.mark.parametrize("dtype,half", [(0, 2 * FF), (1, 2 * FF), (2, 4 * FF)])
@pytest.mark.parametrize("what", ["stride", "wide", "type"])
def test_forward(L, dtype, half, what):  # noqa: F811
    other = (dtype + 1) % 3
    kw = {"stride": dict(h=(P + half, 0), h_dtype=dtype), "wide": dict(a=(P, 136), h=(P + half, 144), h_dtype=dtype),
          "type": dict(h=(P + half, 128), h_dtype=other)}[what]
    d = swiglu(a_dtype=dtype, **kw)
    refused(L, L.tq_swiglu(ctypes.byref(d), None), 1, b"h in place of a's second half")


@pytest.mark.parametrize("dtype,half", [(0, 2 * FF), (1, 2 * FF), (2, 4 * FF)])
def test_gradient(L, dtype, half):  # noqa: F811
    d = swiglu(a_dtype=dtype, h_dtype=dtype, h=(P + half, 72))
    refused(L, L.tq_swiglu_grad(ctypes.byref(d), None), 1, b"h in place of a's second half")
    for ld in (0, 128):             # da's second half, whatever the stride
        d = swiglu(a_dtype=dtype, h_dtype=dtype, da=Q, h=(Q + half, ld))
        refused(L, L.tq_swiglu_grad(ctypes.byref(d), None), 1, b"operands")
        d = swiglu(a_dtype=dtype, h_dtype=dtype, da=(P, 0), h=(P + half, 128 if ld else 136))
        refused(L, L.tq_swiglu_grad(ctypes.byref(d), None), 1, b"operands" if ld else b"h in place of a's second half")
