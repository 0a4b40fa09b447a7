"""Outputs in place of inputs where there is one row: its stride has no meaning
(a slice of one row is dense to torch, whatever lies beside it), so it is never
a reason to refuse the call."""
import ctypes

import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import DT, gen, normal
from tests.test_abi_layer_ops import L, P, combine, swiglu  # noqa: F401  (L: fixture)


def test_no_rows_on_the_host(L):  # noqa: F811
    """No launch follows: only the checks run."""
    assert L.tq_swiglu(ctypes.byref(swiglu(rows=0, a=(P, 0), h=(P, 0))), None) == 0, L.tq_last_error()
    assert L.tq_swiglu(ctypes.byref(swiglu(rows=0, a=(P, 0), h=(P + 128, 0))), None) == 0, L.tq_last_error()
    assert L.tq_swiglu_grad(ctypes.byref(swiglu(rows=0, da=(P, 136))), None) == 0, L.tq_last_error()
    assert L.tq_combine(ctypes.byref(combine(T=0, y=(P, 64), add=(P, 72), w=None)), None) == 0, L.tq_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("ff", [8, 144, 14336])
def test_swiglu(dtype, ff):
    need_gpu()
    a = normal(gen(1), (1, 2 * ff), 2.0, DT[dtype]).cuda()
    h = torch.empty((1, ff), dtype=DT[dtype], device="cuda")
    tq.swiglu(a, h)
    for half in (0, 1):
        b = a.clone()
        tq.swiglu(b, b[:, half * ff:(half + 1) * ff])
        assert torch.equal(b[:, half * ff:(half + 1) * ff], h)
        assert torch.equal(b[:, (1 - half) * ff:(2 - half) * ff], a[:, (1 - half) * ff:(2 - half) * ff])
    # a row of a wider matrix, and the first of several rows
    wide = torch.zeros((3, 2 * ff + 8), dtype=DT[dtype], device="cuda")
    wide[:1, :2 * ff] = a
    tq.swiglu(wide[:1, :2 * ff], wide[:1, :ff])
    assert torch.equal(wide[:1, :ff], h) and torch.equal(wide[:1, ff:2 * ff], a[:, ff:]) and (wide[1:] == 0).all()


@pytest.mark.gpu
def test_gradient_sum_and_layer():
    need_gpu()
    a, dh = normal(gen(2), (1, 288), 1.0, torch.float16).cuda(), normal(gen(3), (1, 144), 1.0, torch.float16).cuda()
    da, h = torch.empty_like(a), torch.empty_like(dh)
    tq.swiglu_grad(a, dh, da, h=h)
    tq.swiglu_grad(a, dh, a, h=dh)
    assert torch.equal(a, da) and torch.equal(dh, h)
    z = normal(gen(4), (2, 144), 1.0, torch.float16).cuda()
    inv, y = torch.tensor([1, 0], dtype=torch.int32, device="cuda"), torch.empty_like(h)
    tq.combine(z, inv, y, add=h)
    tq.combine(z, inv, h, add=h)
    assert torch.equal(y, h)
