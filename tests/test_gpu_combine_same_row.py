"""Rows that several slots name: the sum counts them for each, their dw is that of
each slot, and each value of such a row of dz is that of one of its slots (dz is
the gradient where one slot names a row)."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import check, gen, half_step, normal

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


# a wave a slot; a wave a token
@pytest.mark.parametrize("T,k,d", [(40, 3, 264), (300, 8, 2056), (4100, 4, 136)])
def test_rows_named_more_than_once(T, k, d):
    need_gpu()
    g = gen(21)
    rows = T * k // 4
    inv = torch.randint(0, rows, (T * k,), generator=g, dtype=torch.int32)
    inv[:2] = 5                                 # twice in one token
    z, dy, w = normal(g, (rows, d), 1.0, torch.bfloat16), normal(g, (T, d), 1.0, torch.bfloat16), torch.rand((T, k), generator=g)
    y, dw = torch.empty((T, d), device="cuda"), torch.empty((T, k), device="cuda")
    dz = torch.full((rows, d), -7.0, device="cuda", dtype=torch.bfloat16)
    tq.combine(z.cuda(), inv.cuda(), y, w=w.cuda())
    tq.combine_grad(dy.cuda(), inv.cuda(), w=w.cuda(), z=z.cuda(), dz=dz, dw=dw)
    r, t = inv.long(), torch.arange(T * k) // k
    f = z.double()[r] * w.double().view(-1, 1)
    ref, mag = f.view(T, k, d).sum(1), f.abs().view(T, k, d).sum(1)
    check("y", y, ref, 1.01 * (k + 1) * U * mag + half_step(ref, torch.float32))
    p = z.double()[r] * dy.double()[t]
    check("dw", dw.view(-1), p.sum(1), (d / 64 + 16) * U * p.abs().sum(1))
    one = (w.view(-1, 1) * dy.float()[t]).to(torch.bfloat16)        # (one rounding to f32, one to bf16, as in the kernel)
    got, found = dz.cpu(), torch.zeros((rows, d), dtype=torch.bool)
    found |= (~torch.bincount(r, minlength=rows).bool())[:, None] & (got == -7)
    for s in range(T * k):
        found[r[s]] |= got[r[s]] == one[s]
    assert found.all()
