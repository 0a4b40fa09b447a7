"""Grouping of no tokens: offsets of zero, whatever was in them, so that the
grouped calls that follow take no row."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["current", "stream", "handle", "captured"])
def test_no_tokens(how):
    need_gpu()
    K, k, rows, d, o = 5, 2, 6, 64, 32
    ids = torch.empty((0, k), dtype=torch.int32, device="cuda")
    perm, inv = (torch.empty(0, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.full((tq.group_slots_workspace(0, k, K),), 255, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 1, 2, 3, 5, 6], dtype=torch.int32, device="cuda")     # of the batch before
    # a batch padded to six rows, none of them in use
    dy, x = torch.ones((rows, o), dtype=torch.float16, device="cuda"), torch.ones((rows, d), dtype=torch.float16, device="cuda")
    dw, y = torch.full((K, o, d), 3.0, device="cuda"), torch.full((rows, o), -7.0, device="cuda")
    w = torch.ones((K, o, d), dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step(stream):
        tq.group_slots(ids, K, off, perm, inv, ws, stream=stream)
        tq.group_gemm(x, w, y, off=off, stream=stream)
        tq.group_gemm_dw(dy, x, dw, off=off, stream=stream)

    if how == "captured":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(None)
        for _ in range(3):
            off.fill_(rows)
            dw.fill_(3.0)
            ws.fill_(255)
            torch.randn(1000, device="cuda").sum().item()
            graph.replay()
            torch.cuda.synchronize()
            assert (off == 0).all() and (dw == 0).all() and (y == -7).all() and (ws[:4] == 0).all()
        return
    step({"current": None, "stream": side, "handle": side.cuda_stream}[how])
    torch.cuda.synchronize()
    assert (off == 0).all() and (ws[:4] == 0).all()
    assert (y == -7).all() and (dw == 0).all()
