"""SwiGLU between the products of a layer, its quantised form and its gradient,
against the formulas in 64 bits and against differences.

Bounds, in units of 2^-24 of the value.  The hardware's base-2 exponential and
reciprocal are within an ulp (2 units); the exponent's product is carried to 48
bits, so e^-g has 2 units from the exponential and 1 of the fma that adds the
remainder, plus less than 1 of the remainder's own product; 1 + e^-g 1 more,
where e^-g counts at most fully; the reciprocal 2; g s and its product with up 1
each: 9 in all for h, and 8 for gate s.  The derivative s (1 + g (1 - s)) is s +
(g s)(1 - s): s has 7, 1 - s has 7 of s and 1 of itself, the fma 1; dh up 1 and
the last product 1.  Below -88 the sigmoid is 0, off by less than 2^-126."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.int8_cases import ref_scale
from tests.ops_util import DT, check, gen, half_step, normal

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def reference(a):
    """h and its bound before rounding, in 64 bits."""
    g, u = a.double().chunk(2, dim=1)
    h = g * torch.sigmoid(g) * u
    return h, 9.5 * U * h.abs() + 2.0 ** -125 * (g * u).abs()


def inputs(rows, ff, dtype, seed, wide=0, scale=3.0):
    return normal(gen(seed), (rows, 2 * ff + wide), scale, DT[dtype])


SIZES = [(1, 8), (1, 16), (3, 136), (128, 1408), (67, 2056), (5, 14336), (1000, 24)]


@pytest.mark.parametrize("rows,ff", SIZES)
@pytest.mark.parametrize("adt,hdt", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "f16"),
                                     ("f16", "bf16")])
@pytest.mark.parametrize("wide", [0, 8])
def test_forward(rows, ff, adt, hdt, wide):
    print(f"[case] swiglu {rows} {ff} {adt} {hdt} {wide}", flush=True)
    a = inputs(rows, ff, adt, 1, wide)
    h = torch.full((rows, ff + wide), -7.0, dtype=DT[hdt], device="cuda")
    tq.swiglu(a.cuda()[:, :2 * ff], h[:, :ff])
    ref, tol = reference(a[:, :2 * ff])
    check("h", h[:, :ff], ref, tol + half_step(ref, DT[hdt]))
    assert (h[:, ff:] == -7).all()


def test_the_whole_range_of_the_sigmoid():
    g = torch.cat([torch.linspace(-130, 130, 4001), torch.linspace(-1, 1, 2001), torch.tensor(
        [0.0, -0.0, 1e-38, -1e-38, 1e30, -1e30, 88.0, -88.0, -88.1, 3e38, -3e38])])
    n = -len(g) % 8
    g = torch.cat([g, torch.zeros(n)])
    a = torch.stack([g, torch.full_like(g, 0.75)]).view(1, -1)
    h = torch.empty((1, len(g)), device="cuda")
    tq.swiglu(a.cuda(), h)
    ref, tol = reference(a)
    check("h", h, ref, tol + half_step(ref, torch.float32))
    a = torch.tensor([[float("inf"), float("nan"), 2.0, 2.0, 0.0, 1.0, 1.0, 1.0,
                       1.0, 1.0, float("inf"), float("nan"), 1.0, 1.0, 1.0, 1.0]])
    h = torch.empty((1, 8), device="cuda")
    tq.swiglu(a.cuda(), h)
    h = h.cpu()[0]
    assert h[0] == float("inf") and torch.isnan(h[1]) and h[2] == float("inf") and torch.isnan(h[3]) and h[4] == 0
    assert torch.isfinite(h[5:]).all()


def gradient_reference(a, dh):
    g, u = a.double().chunk(2, dim=1)
    dh = dh.double()
    s = torch.sigmoid(g)
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    mag = (dh * u).abs() * (7 * s + (g * s).abs() * ((8 + 8) * (1 - s) + 7 * s) + 3 * (s * (1 + g * (1 - s))).abs())
    tail = 2.0 ** -125 * (dh.abs() * (1 + u.abs()) * (1 + g.abs()))
    return torch.cat([dg, du], 1), torch.cat([1.05 * U * mag + tail, 9.5 * U * du.abs() + tail], 1)


@pytest.mark.parametrize("rows,ff", SIZES)
@pytest.mark.parametrize("adt,hdt", [("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("again", [True, False])
def test_gradient(rows, ff, adt, hdt, again):
    print(f"[case] swiglu grad {rows} {ff} {adt} {hdt} {again}", flush=True)
    wide = 8 if again else 0
    a, dh = inputs(rows, ff, adt, 2, wide), normal(gen(3), (rows, ff + wide), 1.0, DT[hdt])
    da = torch.full((rows, 2 * ff + wide), -7.0, dtype=DT[adt], device="cuda")
    h = torch.full((rows, ff + wide), -7.0, dtype=DT[adt], device="cuda")
    tq.swiglu_grad(a.cuda()[:, :2 * ff], dh.cuda()[:, :ff], da[:, :2 * ff], h=h[:, :ff] if again else None)
    ref, tol = gradient_reference(a[:, :2 * ff], dh[:, :ff])
    check("da", da[:, :2 * ff], ref, tol + half_step(ref, DT[adt]))
    assert (da[:, 2 * ff:] == -7).all() and (h[:, ff:] == -7).all()
    if again:
        f = torch.empty((rows, ff), dtype=DT[adt], device="cuda")
        tq.swiglu(a.cuda()[:, :2 * ff], f)
        assert torch.equal(h[:, :ff], f)
    else:
        assert (h == -7).all()


def test_gradient_against_differences():
    """Central differences of the kernel's own h in f32: of a step e, the error
    is e^2 / 6 of the third derivative (below 0.6 |up| for silu) and an h's error
    over e."""
    rows, ff, e = 4, 64, 2.0 ** -6
    a = inputs(rows, ff, "f32", 4, scale=1.5)
    ones, da = torch.ones((rows, ff), device="cuda"), torch.empty((rows, 2 * ff), device="cuda")
    tq.swiglu_grad(a.cuda(), ones, da)
    for half in (0, 1):
        h = []
        for sign in (1, -1):
            b = a.clone()
            b[:, half * ff:(half + 1) * ff] += sign * e
            out = torch.empty((rows, ff), device="cuda")
            tq.swiglu(b.cuda(), out)
            h.append(out.double().cpu())
        diff = (h[0] - h[1]) / (2 * e)
        up = a[:, ff:].double().abs() + 1
        tol = e * e / 6 * 0.6 * up + 2 * 10.5 * U * (h[0].abs() + h[1].abs() + 1e-3) / (2 * e) + 2 * U * up / e
        check(f"half {half}", da[:, half * ff:(half + 1) * ff], diff, tol)


@pytest.mark.parametrize("rows,ff,lo,hi,total", [(40, 136, 3, 31, 3), (300, 1408, 0, 299, 60), (20, 2064, 20, 20, 4),
                                                 (9, 40, 0, 0, 1)])
def test_rows_of_offsets(rows, ff, lo, hi, total):
    """Only rows off[0] .. off[groups]-1; the others are left as they were."""
    off = torch.linspace(lo, hi, total + 1).to(torch.int32)
    off[0], off[-1] = lo, hi
    a, dh = inputs(rows, ff, "f16", 5), normal(gen(6), (rows, ff), 1.0, torch.float16)
    a[:lo], a[hi:], dh[:lo], dh[hi:] = (float("nan"),) * 4
    h, hg = (torch.full((rows, ff), -7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    da = torch.full((rows, 2 * ff), -7.0, dtype=torch.float16, device="cuda")
    ad, od = a.cuda(), off.cuda()
    tq.swiglu(ad, h, off=od)
    tq.swiglu_grad(ad, dh.cuda(), da, h=hg, off=od)
    ref, tol = reference(a[lo:hi])
    check("h", h[lo:hi], ref, tol + half_step(ref, torch.float16))
    assert torch.equal(h, hg)
    ref, tol = gradient_reference(a[lo:hi], dh[lo:hi])
    check("da", da[lo:hi], ref, tol + half_step(ref, torch.float16))
    outputs = [h, da]
    if ff % 16 == 0:
        q = torch.full((rows, ff), 77, dtype=torch.int8, device="cuda")
        c = torch.full((rows,), -7.0, device="cuda")
        tq.swiglu_int8(ad, q, c, off=od)
        assert (q[:lo] == 77).all() and (q[hi:] == 77).all()
        assert torch.isfinite(c).all() and (c[lo:hi] > 0).all()
        outputs.append(c)
    for t in outputs:
        assert (t[:lo] == -7).all() and (t[hi:] == -7).all()
    # offsets past the rows are clamped
    tq.swiglu(ad, h, off=torch.tensor([-5, 1 << 30], dtype=torch.int32, device="cuda"))
    assert torch.isnan(h[:lo]).all() and torch.isnan(h[hi:]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,ff,wide", [(1, 16, 0), (33, 1024, 8), (130, 1408, 0), (4, 2048, 0), (6, 2064, 8),
                                          (9, 14336, 0), (2, 32800, 0)])
def test_quantised(dtype, rows, ff, wide):
    """The scale is that of an h within its bound; a code stands for its value
    within half a step, the bound of h, and that of the scale."""
    print(f"[case] swiglu int8 {dtype} {rows} {ff} {wide}", flush=True)
    a = inputs(rows, ff, dtype, 7, wide, scale=1.5)
    q, c = torch.empty((rows, ff), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    tq.swiglu_int8(a.cuda()[:, :2 * ff], q, c)
    ref, tol = reference(a[:, :2 * ff])
    amax = ref.abs().amax(1)
    check("scale", c, amax / 127, (tol + 2 * U * ref.abs()).amax(1) / 127 + U * amax / 127)
    cd = c.double().cpu()[:, None]
    check("value", q.double().cpu() * cd, ref, 0.5 * cd + tol + 2 * U * ref.abs())
    assert (q.abs().amax(1) == 127).all() and int(q.min()) >= -127
    # the same as of swiglu's own f32 result, code for code
    h = torch.empty((rows, ff), device="cuda")
    tq.swiglu(a.cuda()[:, :2 * ff], h)
    q2, c2 = torch.empty_like(q), torch.empty_like(c)
    tq.int8_quant_rows(h, q2, c2)
    assert torch.equal(q, q2) and torch.equal(c, c2)


def test_quantised_special_rows():
    a = torch.ones((4, 64))
    a[0, :32] = 0.0                       # h is zero: scale 1
    a[1, 3] = float("nan")
    a[2, 40] = float("inf")
    q, c = torch.full((4, 32), 77, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    tq.swiglu_int8(a.cuda(), q, c)
    c = c.cpu()
    assert c[0] == 1 and torch.isnan(c[1]) and torch.isnan(c[2]) and (q[:3] == 0).all() and (q[3] == 127).all()
    assert (c[3] - ref_scale(torch.sigmoid(torch.tensor(1.0)))).abs() < 1e-8


def test_in_place():
    a, dh = inputs(37, 144, "bf16", 8).cuda(), normal(gen(9), (37, 144), 1.0, torch.bfloat16).cuda()
    h, da, hg = torch.empty_like(dh), torch.empty_like(a), torch.empty_like(dh)
    tq.swiglu(a, h)
    tq.swiglu_grad(a, dh, da, h=hg)
    for half in (0, 1):
        b = a.clone()
        tq.swiglu(b, b[:, 144 * half:144 * (half + 1)])
        assert torch.equal(b[:, 144 * half:144 * (half + 1)], h)
        assert torch.equal(b[:, 144 * (1 - half):144 * (2 - half)], a[:, 144 * (1 - half):144 * (2 - half)])
    b, d = a.clone(), dh.clone()
    tq.swiglu_grad(b, d, b, h=d)
    assert torch.equal(b, da) and torch.equal(d, hg)


def test_graph_and_streams():
    a, dh = inputs(50, 144, "f16", 10).cuda(), normal(gen(11), (50, 144), 1.0, torch.float16).cuda()
    h, da = torch.empty_like(dh), torch.empty_like(a)
    q, c = torch.empty((50, 144), dtype=torch.int8, device="cuda"), torch.empty(50, device="cuda")

    def step(stream=None):
        tq.swiglu(a, h, stream=stream)
        tq.swiglu_grad(a, dh, da, stream=stream)
        tq.swiglu_int8(a, q, c, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (h, da, q, c)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for how in ("stream", "handle", "graph", "graph", "graph"):
        for t in (h, da, q, c):
            t.fill_(3)
        torch.randn(1000, device="cuda").sum().item()
        torch.cuda.synchronize()
        if how == "graph":
            graph.replay()
        else:
            step(side if how == "stream" else side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip((h, da, q, c), want))


def test_no_rows():
    a, h = torch.empty((0, 32), device="cuda"), torch.empty((0, 16), device="cuda")
    tq.swiglu(a, h)
    tq.swiglu_grad(a, h, a.clone())
    tq.swiglu_int8(a, h.to(torch.int8), torch.empty(0, device="cuda"))
