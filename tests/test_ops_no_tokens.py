"""The sum over a token's slots and its gradient for a batch without tokens: inv
as group_slots takes it, [0], names no number of slots, so the weights do (on
the host; the entry is replaced by one that records its arguments)."""
import ctypes

import pytest

import bit_rank_post_amd as tq
from tests.test_abi_layer_ops import F32, I32, meta


@pytest.fixture
def calls(monkeypatch):
    from bit_rank_post_amd import ops
    seen = []
    monkeypatch.setattr(ops, "_device", lambda fn, *t: 0)
    monkeypatch.setattr(ops, "_call", lambda fn, dev, stream, d: seen.append(
        (fn, ctypes.cast(d, ctypes.POINTER(tq.CombineDesc)).contents.topk)))
    return seen


@pytest.mark.parametrize("k", [1, 2, 8])
@pytest.mark.parametrize("inv", [(0,), (0, None)])
def test_without_tokens(calls, k, inv):
    inv = meta(*[k if n is None else n for n in inv], dtype=I32)
    z, y, w, dw = meta(8, 16), meta(0, 16), meta(0, k, dtype=F32), meta(0, k, dtype=F32)
    tq.combine(z, inv, y, w=w)
    tq.combine_grad(y, inv, w=w, z=z, dz=meta(8, 16), dw=dw)
    tq.combine_grad(y, inv, z=z, dw=dw)
    assert calls == [("combine", k), ("combine_grad", k), ("combine_grad", k)]
    tq.combine(z, inv, y)
    tq.combine_grad(y, inv, dz=meta(8, 16))
    assert len(calls) == 5


def test_refused(calls):
    for call in (lambda: tq.combine(meta(8, 16), meta(0, dtype=I32), meta(0, 16), w=meta(1, 2, dtype=F32)),
                 lambda: tq.combine(meta(8, 16), meta(4, dtype=I32), meta(0, 16), w=meta(0, 2, dtype=F32)),
                 lambda: tq.combine(meta(8, 16), meta(0, dtype=I32), meta(0, 16), w=meta(0, dtype=F32)),
                 lambda: tq.combine_grad(meta(0, 16), meta(0, dtype=I32), w=meta(0, 2, dtype=F32), z=meta(8, 16),
                                         dw=meta(0, 3, dtype=F32))):
        with pytest.raises(tq.TileQError, match="is .*must be"):
            call()
    assert not calls
