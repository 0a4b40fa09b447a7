"""The gate's gradient of SwiGLU where dh times up leaves f32 and the gradient
does not: far below zero the slope is small, so no order of the products may
overflow or lose bits on the way.  Bounds as in test_gpu_swiglu_slope; all
values here are normal numbers, their parts too."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import check
from tests.test_gpu_swiglu_slope import U, slope

pytestmark = pytest.mark.gpu

# gate, up, dh
CASES = [(-5.0, 1e30, 1e9), (-5.0, 1e9, 1e30), (-20.0, -3e38, 1e5), (-20.0, 1e5, -3e38), (-60.0, 1e20, 1e30), (-60.0, 1e30, 1e20),
         (0.0, 2e38, 3.0), (0.0, 3.0, -2e38), (-25.0, 1e-30, 1e30), (-25.0, 1e30, 1e-30), (-30.0, 1e-33, 1e38), (-30.0, 1e38, 1e-33),
         (3.0, 1e-20, 1e30), (3.0, 3e38, 0.5), (3.0, 0.5, 3e38), (-1.5, 1e19, 1e20)]


def test_products_stay_in_range():
    need_gpu()
    t = torch.tensor(CASES)
    g, u, dh = (v.view(-1, 1).expand(-1, 8).contiguous() for v in t.unbind(1))
    da = torch.empty((len(CASES), 16), device="cuda")
    tq.swiglu_grad(torch.cat([g, u], 1).cuda(), dh.cuda(), da)
    d, mag = slope(g.double())
    p = u.double() * dh.double()
    ref = d * p
    assert (ref.abs() < 3.3e38).all() and (ref.abs() > 2.0 ** -126).all()
    check("dgate", da[:, :8], ref, 1.05 * U * mag * p.abs())


def test_infinities_and_nan_stay():
    need_gpu()
    inf, nan = float("inf"), float("nan")
    t = torch.tensor([(-1.0, inf, 1.0), (1.0, 1.0, inf), (1.0, nan, 1.0), (1.0, 1.0, nan), (nan, 1.0, 1.0), (1.0, 3e38, 3e38), (1.0, inf, 0.0),
                      (1.0, 0.0, 0.0)])
    g, u, dh = t.unbind(1)
    da = torch.empty((1, 16), device="cuda")
    tq.swiglu_grad(torch.cat([g, u])[None].cuda(), dh[None].cuda(), da)
    got = da[0, :8].cpu()
    # (the slope is 0.07 at -1 and 0.93 at 1)
    assert (got[[0, 1, 5]] == inf).all() and torch.isnan(got[[2, 3, 4, 6]]).all() and got[7] == 0
