"""Offsets past 32 bits: matrices of more than 2^32 bytes, whose last rows, slots
and experts are what is computed, beside the first."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.int8_cases import product, quantised
from tests.ops_util import check, half_step

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()
    yield
    torch.cuda.empty_cache()


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def filled(shape, dtype, seed):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, 1.0, generator=rng(seed))


def test_swiglu_and_quantisation():
    rows, ff = 140000, 8192                     # a: 2.3e9 values
    a = filled((rows, 2 * ff), torch.float16, 1)
    h, q = torch.empty((rows, ff), dtype=torch.float16, device="cuda"), torch.empty((rows, ff), dtype=torch.int8, device="cuda")
    c = torch.empty(rows, device="cuda")
    tq.swiglu(a, h)
    for part in (slice(0, 3), slice(rows - 3, rows), slice(131070, 131074)):
        g, u = a[part].double().chunk(2, 1)
        ref = (g * torch.sigmoid(g) * u).cpu()
        check("h", h[part], ref, 9.5 * 2.0 ** -24 * ref.abs() + half_step(ref, torch.float16))
    tq.swiglu_int8(a, q, c)
    for part in (slice(0, 2), slice(rows - 2, rows)):
        g, u = a[part].double().chunk(2, 1)
        ref, cd = (g * torch.sigmoid(g) * u).cpu(), c[part].double().cpu()[:, None]
        check("q c", q[part].double() * cd.cuda(), ref, 0.5 * cd + 12 * 2.0 ** -24 * ref.abs())
    del h, q
    q, c = torch.empty((rows, 2 * ff), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    tq.int8_quant_rows(a, q, c)
    for part in (slice(0, 2), slice(rows - 2, rows)):
        rq, rc = quantised(a[part].cpu())
        assert torch.equal(q[part].cpu(), rq) and torch.equal(c[part].cpu(), rc)
    # the gradient in place of a
    last = a[-2:].clone()
    dh = filled((2, ff), torch.float16, 2)
    want = torch.empty_like(last)
    tq.swiglu_grad(last, dh, want)
    all_dh = torch.zeros((rows, ff), dtype=torch.float16, device="cuda")
    all_dh[-2:] = dh
    tq.swiglu_grad(a, all_dh, a)
    assert torch.equal(a[-2:], want) and (a[:100] == 0).all()


def test_combine():
    T, k, d = 70000, 4, 8192                    # z: 2.3e9 values
    z = filled((T * k, d), torch.float16, 3)
    inv = torch.arange(T * k - 1, -1, -1, dtype=I32, device="cuda")
    y = torch.empty((T, d), dtype=torch.float16, device="cuda")
    tq.combine(z, inv, y)
    for t in (0, T - 1, 32768):
        rows = z[inv[t * k:(t + 1) * k].long()].double().cpu()
        ref = rows.sum(0)
        check(f"token {t}", y[t], ref, 5.1 * 2.0 ** -24 * rows.abs().sum(0) + half_step(ref, torch.float16))
    w, dw = torch.rand((T, k), device="cuda", generator=rng(4)), torch.empty((T, k), device="cuda")
    keep = {t: z[inv[t * k:(t + 1) * k].long()].double().cpu() for t in (0, T - 1)}
    tq.combine_grad(y, inv, w=w, z=z, dz=z, dw=dw)            # dz in place of z
    for t, rows in keep.items():
        dy = y[t].double().cpu()
        check(f"dw {t}", dw[t], (rows * dy).sum(1), (d / 64 + 16) * 2.0 ** -24 * (rows * dy).abs().sum(1))
        ref = w[t].double().cpu()[:, None] * dy
        check(f"dz {t}", z[inv[t * k:(t + 1) * k].long()], ref, 1.01 * 2.0 ** -24 * ref.abs() + half_step(ref, torch.float16))


@pytest.mark.parametrize("rows", [6, 400])
def test_int8_product(rows):
    G, o, i = 34, 8192, 16384                   # w: 4.6e9 codes
    w = torch.randint(-128, 128, (G, o, i), dtype=torch.int8, device="cuda", generator=rng(5))
    ws, x = torch.rand((G, o), device="cuda", generator=rng(6)), torch.randint(-128, 128, (rows, i), dtype=torch.int8, device="cuda", generator=rng(7))
    xs, y = torch.rand(rows, device="cuda", generator=rng(8)), torch.empty((rows, o), device="cuda")
    off = torch.full((G + 1,), rows // 2, dtype=I32, device="cuda")
    off[0], off[G] = 0, rows                    # the first and the last expert
    tq.int8_gemm(x, xs, w, ws, y, off=off)
    for e, part in ((0, slice(0, 2)), (G - 1, slice(rows - 2, rows))):
        want = product(x[part].cpu(), xs[part].cpu(), w[e].cpu(), ws[e].cpu(), torch.float32)
        assert torch.equal(y[part].cpu(), want)


@pytest.mark.parametrize("T", [1, 3, 20])
def test_layer(T):
    E, k, d, ff = 36, 2, 8192, 4096             # w_up: 2.4e9 values
    w_up, w_down = filled((E, 2 * ff, d), torch.float16, 9).mul_(d ** -0.5), filled((E, d, ff), torch.float16, 10).mul_(ff ** -0.5)
    x = filled((T, d), torch.float16, 11)
    ids = torch.tensor([[E - 1, 0]] * T, dtype=I32, device="cuda")
    w, y = torch.rand((T, k), device="cuda", generator=rng(12)), torch.empty((T, d), device="cuda")
    ws = torch.empty(tq.experts_workspace(T, k, E, d, ff), dtype=torch.uint8, device="cuda")
    tq.experts_forward(x, ids, w, w_up, w_down, y, ws)
    ref, tol = torch.zeros((T, d), dtype=torch.float64), torch.zeros((T, d), dtype=torch.float64)
    xd = x.double().cpu()
    for j, e in enumerate((E - 1, 0)):
        u, v, c = w_up[e].double().cpu(), w_down[e].double().cpu(), w[:, j].double().cpu()[:, None]
        g, up = (xd @ u.t()).chunk(2, 1)
        ea = (d + 1) * 2.0 ** -23 * (xd.abs() @ u.abs().t())
        eg, eu = ea.chunk(2, 1)
        h = g * torch.sigmoid(g) * up
        eh = 1.1 * eg * up.abs() + g.abs() * eu + 1.1 * eg * eu + 2.0 ** -20 * h.abs()
        eh = eh + 2 * half_step(h.abs() + eh, torch.float16)
        h = h.half().double()
        ref += c * (h @ v.t())
        tol += c * ((ff + k + 4) * 2.0 ** -23 * (h.abs() @ v.abs().t()) + eh @ v.abs().t())
    check("y", y, ref, 1.01 * tol)
