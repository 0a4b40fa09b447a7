"""The layer for a few tokens addresses x with 32-bit offsets: strides that take
it past 2^31 bytes are refused, also those whose product with the rows does not
fit 64 bits (host only)."""
import ctypes

import pytest

from tests.test_abi_layer_ops import L, P, R, experts, refused  # noqa: F401  (L: fixture)


@pytest.mark.parametrize("T", [1, 2, 4, 5, 512])
@pytest.mark.parametrize("ld", [1 << 30, 1 << 31, 1 << 32, 1 << 52, 1 << 60, 1 << 61, 1 << 62, (1 << 63) - 8])
def test_refused(L, T, ld):  # noqa: F811
    d = experts(T=T, x=(R, ld))
    refused(L, L.tq_experts_forward(ctypes.byref(d), P, 0, None), 5, b"2^31")


@pytest.mark.parametrize("T", [1, 3, 4, 512])
def test_the_border(L, T):  # noqa: F811
    """The largest stride that is taken: the next check, a workspace too small, is
    reached."""
    ld = 0x7FFFFFEF // 2 // T // 8 * 8
    refused(L, L.tq_experts_forward(ctypes.byref(experts(T=T, x=(R, ld))), P, 0, None), 2, b"ws_bytes")
    assert ld * 2 * T < 0x7FFFFFF0
    ld = -(-0x7FFFFFF0 // 2 // T)
    ld = -(-ld // 8) * 8
    refused(L, L.tq_experts_forward(ctypes.byref(experts(T=T, x=(R, ld))), P, 0, None), 5, b"2^31")
