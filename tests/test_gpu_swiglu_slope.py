"""The gate's gradient of SwiGLU, dh u s (1 + g (1 - s)), in f32, where nothing of
a rounding to 16 bits covers its error.

Bound in units of 2^-24 of each part's value.  e = e^-g has 4: 2 of the hardware's
exponential (an ulp), 1 of the fma that adds the remainder of the exponent, less
than 1 of that remainder.  s = 1 / (1 + e): of e's 4 the part 1 - s, 1 of the sum,
2 of the reciprocal (an ulp).  1 - s = e s: of e's 4 the part s, 3 as s, 1 of the
product.  g s (1 - s): 4 at most of e (the parts are s and 1 - s, of opposite
signs), 3 twice, 1 of each of its two products: 12.  The slope is s + g s (1 - s)
by one fma: s (3 + 4 (1 - s)) + 12 |g s (1 - s)| and 1 of the slope; its products
with dh and u 2 more.  (1.05: terms of second order.)  Where s leaves the normal
numbers it may be off by 2^-126."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import check, gen

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def slope(g):
    """s (1 + g (1 - s)) in 64 bits and its bound, without the products with dh and u."""
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    d = s + g * s * r
    return d, s * (3 + 4 * r) + 12 * (g * s * r).abs() + 3 * d.abs()


@pytest.mark.parametrize("lo,hi", [(-4.0, 4.0), (2.0, 24.0), (-90.0, 0.0), (16.0, 130.0)])
@pytest.mark.parametrize("ones", [True, False])
def test_the_slope(lo, hi, ones):
    n = 1 << 16
    g = torch.linspace(lo, hi, n).view(64, -1)
    ff = g.shape[1]
    u, dh = torch.ones_like(g), torch.ones_like(g)
    if not ones:
        u, dh = torch.randn(g.shape, generator=gen(1)), torch.randn(g.shape, generator=gen(2)) * 30
    da = torch.empty((64, 2 * ff), device="cuda")
    tq.swiglu_grad(torch.cat([g, u], 1).cuda(), dh.cuda(), da)
    d, mag = slope(g.double())
    p = u.double() * dh.double()
    tail = 2.0 ** -125 * (1 + g.double().abs()) * (1 + p.abs()) * 2
    check("dgate", da[:, :ff], d * p, 1.05 * U * mag * p.abs() + tail)


def test_far_gates():
    """The sigmoid is 0 or 1 there, and so is the slope, whatever the gate."""
    g = torch.tensor([[88.0, 88.1, 89.0, 104.0, 1e4, 1e30, 3e38, 88.0], [-88.0, -88.1, -89.0, -104.0, -1e4, -1e30, -3e38, -87.5]])
    a = torch.cat([g, torch.ones_like(g)], 1)
    da = torch.empty((2, 16), device="cuda")
    tq.swiglu_grad(a.cuda(), torch.ones((2, 8), device="cuda"), da)
    assert (da[0, :8] == 1).all() and torch.equal(da[0, 8:].cpu(), g[0])
    assert (da[1, :8].abs() < 100 * 2.0 ** -125).all() and (da[1, 8:].abs() <= 2.0 ** -126 * g[1].abs().cuda()).all()
