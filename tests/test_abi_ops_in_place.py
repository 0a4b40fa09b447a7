"""Outputs in place of inputs with another row stride are refused (host only):
a row would be written where one lies that is not read yet."""
import ctypes

import pytest

from tests.test_abi_ops import L, P, grad, norm  # noqa: F401  (L: fixture)


@pytest.mark.parametrize("kw,text", [
    (dict(x=(P, 128), y=(P, 64)), b"y in place of x"), (dict(x=(P, 64), y=(P, 128)), b"y in place of x"),
    (dict(b=(P, 0), n=(P, 72)), b"n in place of b"), (dict(b=(P, 72), n=(P, 80)), b"n in place of b"),
])
def test_norm(L, kw, text):  # noqa: F811
    assert L.tq_norm_residual(ctypes.byref(norm(**kw)), None) == 1, L.tq_last_error()
    assert text in L.tq_last_error(), L.tq_last_error()


@pytest.mark.parametrize("kw,text", [
    (dict(dx=(P, 72)), b"dx in place of dy"), (dict(dy=(P + 4096, 0), dx=(P, 72)), b"dx in place of y"),
    (dict(db=(P, 72)), b"db in place of dn"), (dict(dn=(P + 4096, 0), db=(P, 72)), b"db in place of b"),
    (dict(dn=(P, 128), db=(P, 64)), b"db in place of dn"),
])
def test_gradients(L, kw, text):  # noqa: F811
    assert L.tq_norm_residual_grad(ctypes.byref(grad(**kw)), P, 1 << 30, None) == 1, L.tq_last_error()
    assert text in L.tq_last_error(), L.tq_last_error()
