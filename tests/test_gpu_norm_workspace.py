"""The norm gradients' own workspace on explicit streams and in captures."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.norm_cases import prepared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


@pytest.mark.parametrize("how", ["stream", "handle", "null handle"])
def test_own_workspace_on_another_stream(how):
    """Without ws, the workspace belongs to the stream of the call."""
    T, d = 900, 1032
    s, y, kw, out = prepared(T, d, ("bf16", "bf16", "bf16"), "token", 10)
    tq.norm_residual_grad(y, dy=s["dy"], dn=s["dn"], **kw, **out)
    want = {k: v.clone() for k, v in out.items()}
    side = torch.cuda.Stream()
    other = torch.empty(1 << 20, device="cuda")
    for _ in range(5):
        for v in out.values():
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        stream = {"stream": side, "handle": side.cuda_stream, "null handle": 0}[how]
        tq.norm_residual_grad(y, dy=s["dy"], dn=s["dn"], stream=stream, **kw, **out)
        other = other * 2.0 + 1.0          # work and allocations of the current stream meanwhile
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in out)


@pytest.mark.parametrize("handle", [False, True])
def test_own_workspace_in_a_capture_on_an_explicit_stream(handle):
    T, d = 900, 1032
    s, y, kw, out = prepared(T, d, ("bf16", "bf16", "bf16"), "token", 11)
    tq.norm_residual_grad(y, dy=s["dy"], dn=s["dn"], **kw, **out)
    want = {k: v.clone() for k, v in out.items()}
    side, current = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(current):       # the captured stream is not the current one
            tq.norm_residual_grad(y, dy=s["dy"], dn=s["dn"], stream=side.cuda_stream if handle else side, **kw, **out)
    for _ in range(4):
        for v in out.values():
            v.fill_(float("nan"))
        torch.randn(1 << 20, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in out)
