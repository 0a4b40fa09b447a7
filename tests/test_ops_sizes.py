"""Sizes past 32 bits are refused by the torch functions (host only: the tensors
have shapes and no memory, and no call reaches the library)."""
import pytest
import torch

import bit_rank_post_amd as tq
from bit_rank_post_amd import ops

BIG = (1 << 32) + 4
E4M3 = torch.float8_e4m3fn


def empty(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(ops, "_device", lambda fn, *t: 0)

    def reached(fn, *a):
        raise AssertionError(f"{fn} would have been called")

    monkeypatch.setattr(ops, "_call", reached)


F32 = torch.float32
I32 = torch.int32


class FakeLayer:
    act, d_model, K, h = tq.TQ_F16, 16, 8, None


@pytest.mark.parametrize("call", [
    lambda: tq.group_gemm(empty(BIG, 16), empty(8, 16), empty(BIG, 8)),
    lambda: tq.group_gemm(empty(4, 16), empty(8, 16), empty(4, 8), src=empty(4, dtype=I32), src_div=BIG),
    lambda: tq.group_gemm(empty(4, 16), empty(8, 16), empty(4, 8), src=empty(4, dtype=I32), src_div=-BIG),
    lambda: tq.group_gemm(empty(BIG, 16), empty(8, 16), empty(4, 8), src=empty(4, dtype=I32)),
    lambda: tq.group_gemm_dx(empty(BIG, 8), empty(8, 16), empty(BIG, 16)),
    lambda: tq.group_gemm_dw(empty(BIG, 8), empty(BIG, 16), empty(8, 16)),
    lambda: tq.group_gemm_dw(empty(4, BIG), empty(4, 16), empty(BIG, 16)),
    lambda: tq.fp8_gemm(empty(BIG, 16, dtype=E4M3), empty(BIG, 1, dtype=F32), empty(8, 16, dtype=E4M3),
                        empty(1, 1, dtype=F32), empty(BIG, 8)),
    lambda: tq.fp8_quant_rows(empty(BIG, 16), empty(BIG, 16, dtype=E4M3), empty(BIG, 1, dtype=F32)),
    lambda: tq.fp8_quant_blocks(empty(BIG, 16), empty(BIG, 16, dtype=E4M3),
                                empty(-(-BIG // 128), 1, dtype=F32)),
    lambda: tq.norm_residual(empty(BIG, 8), n=empty(BIG, 8), w_next=empty(8)),
    lambda: tq.norm_residual(empty(4, BIG), n=empty(4, BIG), w_next=empty(BIG)),
    lambda: tq.norm_residual_grad(empty(BIG, 8), dx=empty(BIG, 8), dy=empty(BIG, 8)),
    lambda: ops.norm_grad_workspace(BIG, 8),
    lambda: tq.group_slots_workspace(BIG, 2, 8),
    lambda: tq.group_slots(empty(BIG, 1, dtype=I32), 8, empty(9, dtype=I32), empty(BIG, dtype=I32),
                           empty(BIG, dtype=I32), empty(512, dtype=torch.uint8)),
    lambda: ops.block_forward(FakeLayer, empty(BIG, 16), empty(BIG, 16), empty(8, 16), empty(16), 2,
                              empty(BIG, 2, dtype=I32), empty(BIG, 2, dtype=F32), empty(512, dtype=torch.uint8)),
])
def test_refused(call):
    with pytest.raises(tq.TileQError, match="does not fit 32 bits"):
        call()
