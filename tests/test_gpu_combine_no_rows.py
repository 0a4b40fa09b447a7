"""The gradient of the sum over slots where there are no rows (all slots of a
batch were dropped, or an expert-parallel rank got none): dz has nothing to
take, dw is 0."""
import ctypes

import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.test_abi_layer_ops import L, P, combine, refused  # noqa: F401  (L: fixture)


def test_nothing_to_write_on_the_host(L):  # noqa: F811
    """No launch follows."""
    for kw in (dict(z=None, dz=None), dict(dz=None), dict(z=None)):
        d = combine(rows=0, dw=None, **kw)
        assert L.tq_combine_grad(ctypes.byref(d), None) == 0, L.tq_last_error()
    # with rows it is a mistake, and the other checks still run
    refused(L, L.tq_combine_grad(ctypes.byref(combine(dz=None, dw=None)), None), 1, b"neither")
    refused(L, L.tq_combine_grad(ctypes.byref(combine(rows=0, dw=None, dz=None, dy=None)), None), 1, b"dy is NULL")
    refused(L, L.tq_combine_grad(ctypes.byref(combine(rows=0, dw=None, dz=None, inv=None)), None), 1, b"inv is NULL")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 5000])
def test_no_rows(T):
    need_gpu()
    k, d = 2, 64
    inv = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    inv[1] = 0
    dy, w, z = torch.randn((T, d), device="cuda"), torch.rand((T, k), device="cuda"), torch.empty((0, d), device="cuda")
    tq.combine_grad(dy, inv, w=w, dz=z)
    tq.combine_grad(dy, inv, z=z, dz=z)
    dw = torch.full((T, k), 7.0, device="cuda")
    tq.combine_grad(dy, inv, w=w, z=z, dz=torch.empty_like(z), dw=dw)
    assert (dw == 0).all()
