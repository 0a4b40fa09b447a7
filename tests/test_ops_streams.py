"""A stream of another device than the operands' is refused (host only)."""
import pytest

import bit_rank_post_amd as tq
from bit_rank_post_amd import ops


class Stream:
    cuda_stream = 0x1000

    def __init__(self, device):
        self.device_index = device


def test_stream_of_another_device(monkeypatch):
    called = []
    monkeypatch.setitem(ops._entries, "norm_residual", lambda *a: called.append(a) or 0)
    monkeypatch.setattr(ops.torch.cuda, "current_device", lambda: 1)
    with pytest.raises(tq.TileQError, match="a stream of cuda:0 for operands on cuda:1"):
        ops._call("norm_residual", 1, Stream(0), "descriptor")
    assert not called
    ops._call("norm_residual", 1, Stream(1), "descriptor")
    ops._call("norm_residual", 1, 0x2000, "descriptor")          # a raw handle says nothing about its device
    assert called == [("descriptor", 0x1000), ("descriptor", 0x2000)]
