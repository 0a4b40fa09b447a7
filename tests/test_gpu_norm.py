"""Norms around a block and their gradients against the formulas in 64 bits,
and the gradients against differences of the forward formula."""
import itertools

import pytest
import torch

import bit_rank_post_amd as tq
from bit_rank_post_amd import ops
from tests.gpu_util import need_gpu
from tests.ops_util import DT, check, gen, half_step, normal

pytestmark = pytest.mark.gpu
EPS, U = 1e-6, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


SIZES = [(1, 8), (1, 4096), (3, 64), (5, 512), (7, 520), (66, 2048), (4, 4104), (130, 2056), (2, 8200), (9, 16384),
         (700, 128)]
TYPES = [("f16", "f16", "f16"), ("bf16", "bf16", "f32"), ("f32", "bf16", "bf16"), ("f32", "f32", "f32"),
         ("bf16", "f16", "f16"), ("f16", "f32", "bf16")]


def inputs(T, d, sdt, adt, wdt, gate, seed=1):
    g = gen(seed)
    s = dict(x=normal(g, (T, d), 2.0, DT[sdt]), b=normal(g, (T, d), 0.7, DT[adt]),
             w_post=(1 + normal(g, (d,), 0.2, torch.float32)).to(DT[wdt]),
             w_next=(1 + normal(g, (d,), 0.2, torch.float32)).to(DT[wdt]), gate=None,
             dy=normal(g, (T, d), 1.0, DT[sdt]), dn=normal(g, (T, d), 1.0, DT[adt]))
    if gate == "token":
        s["gate"] = torch.sigmoid(normal(g, (T,), 1.0, torch.float32))
    if gate == "full":
        s["gate"] = torch.sigmoid(normal(g, (T, d), 1.0, torch.float32)).to(DT[adt])
    return s


def col(g):
    return 1.0 if g is None else g.double().view(g.shape[0], -1)


def forward_ref(s, alpha, post=True):
    b, x = s["b"].double(), s["x"].double()
    r1 = (b.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    p = b * r1 * s["w_post"].double() if post else b
    return x + alpha * col(s["gate"]) * p, r1, (alpha * col(s["gate"]) * p).abs() + x.abs()


def norm_ref(y, w):
    r2 = (y.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    return y * r2 * w.double(), r2


# relative error of r = (mean + eps)^-1/2 in f32: a sum of d squares in any
# order is within d U (each square adds U), the division, sum with eps and the
# root's approximation 4 U more; half of it passes through the root
def r_tol(d):
    return (d + 1) * U / 2 + 4 * U


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("sdt,adt,wdt", TYPES)
@pytest.mark.parametrize("gate", ["none", "token", "full"])
def test_forward(T, d, sdt, adt, wdt, gate):
    print(f"[case] norm forward {T} {d} {sdt} {adt} {wdt} {gate}", flush=True)
    s = inputs(T, d, sdt, adt, wdt, gate)
    c = {k: (v.cuda() if v is not None else None) for k, v in s.items()}
    y, n = torch.empty_like(c["x"]), torch.empty_like(c["b"])
    rp, rn = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    tq.norm_residual(c["x"], y=y, n=n, b=c["b"], w_post=c["w_post"], w_next=c["w_next"], gate=c["gate"],
                     alpha=0.75, eps=EPS, rstd_post=rp, rstd_next=rn)
    ref, r1, mag = forward_ref(s, 0.75)
    check("r1", rp, r1[:, 0], r_tol(d) * r1[:, 0])
    # p: r1, two products, alpha gate and the fused sum
    check("y", y, ref, (r_tol(d) + 6 * U) * mag + half_step(ref, DT[sdt]))
    # n and r2 are those of the y that was stored
    stored = y.double().cpu()
    ref, r2 = norm_ref(stored, s["w_next"])
    check("r2", rn, r2[:, 0], r_tol(d) * r2[:, 0])
    check("n", n, ref, (r_tol(d) + 3 * U) * ref.abs() + half_step(ref, DT[adt]))


@pytest.mark.parametrize("T,d", [(1, 4096), (33, 136), (5, 8192), (300, 1408)])
def test_parts_of_the_forward(T, d):
    """The norm alone, the residual alone, without the post-norm, and y in
    place of x, n in place of b: the same values as the whole."""
    s = inputs(T, d, "bf16", "bf16", "bf16", "token", seed=2)
    c = {k: v.cuda() for k, v in s.items()}
    y, n = torch.empty_like(c["x"]), torch.empty_like(c["b"])
    tq.norm_residual(c["x"], y=y, n=n, b=c["b"], w_post=c["w_post"], w_next=c["w_next"], gate=c["gate"], alpha=0.5)
    y2, n2 = torch.empty_like(y), torch.empty_like(n)
    tq.norm_residual(c["x"], y=y2, b=c["b"], w_post=c["w_post"], gate=c["gate"], alpha=0.5)
    tq.norm_residual(y2, n=n2, w_next=c["w_next"])
    assert torch.equal(y, y2) and torch.equal(n, n2)
    xi, bi = c["x"].clone(), c["b"].clone()
    tq.norm_residual(xi, y=xi, n=bi, b=bi, w_post=c["w_post"], w_next=c["w_next"], gate=c["gate"], alpha=0.5)
    assert torch.equal(xi, y) and torch.equal(bi, n)
    tq.norm_residual(c["x"], y=y2, b=c["b"], gate=c["gate"], alpha=-2.0)
    ref, _, mag = forward_ref(s, -2.0, post=False)
    check("without post-norm", y2, ref, 4 * U * mag + half_step(ref, torch.bfloat16))


def test_strides_and_rows_outside():
    T, d = 37, 264
    s = inputs(T, d, "f32", "f16", "f16", "full", seed=3)
    c = {k: v.cuda() for k, v in s.items()}

    def wide(t, fill):
        w = torch.full((T + 2, d + 24), fill, dtype=t.dtype, device="cuda")
        w[1:T + 1, 8:8 + d] = t
        return w, w[1:T + 1, 8:8 + d]

    (_, x), (_, b), (_, g) = wide(c["x"], float("nan")), wide(c["b"], float("nan")), wide(c["gate"], float("nan"))
    (yw, y), (nw, n) = wide(torch.zeros_like(c["x"]), -7.0), wide(torch.zeros_like(c["b"]), -7.0)
    tq.norm_residual(x, y=y, n=n, b=b, w_post=c["w_post"], w_next=c["w_next"], gate=g)
    y2, n2 = torch.empty_like(c["x"]), torch.empty_like(c["b"])
    tq.norm_residual(c["x"], y=y2, n=n2, b=c["b"], w_post=c["w_post"], w_next=c["w_next"], gate=c["gate"])
    assert torch.equal(y, y2) and torch.equal(n, n2)
    for w in (yw, nw):
        inner = w[1:T + 1, 8:8 + d].clone()
        w[1:T + 1, 8:8 + d] = -7
        assert (w == -7).all() and torch.isfinite(inner).all()
    # a strided gate per token
    gt = torch.rand((T, 3), device="cuda")
    tq.norm_residual(c["x"], y=y2, b=c["b"], gate=gt[:, 1])
    tq.norm_residual(c["x"], y=n2.float(), b=c["b"], gate=gt[:, 1].contiguous())
    y3 = torch.empty_like(y2)
    tq.norm_residual(c["x"], y=y3, b=c["b"], gate=gt[:, 1].contiguous())
    assert torch.equal(y2, y3)


def test_special_rows():
    """Zero rows, huge rows and rows with NaN or infinity stay by themselves."""
    T, d = 6, 1024
    x = torch.ones((T, d), dtype=torch.float32, device="cuda")
    x[0], x[1], x[2, 5], x[3, 9] = 0, 3e4, float("nan"), float("inf")
    w = torch.full((d,), 2.0, device="cuda")
    n = torch.empty((T, d), device="cuda")
    tq.norm_residual(x, n=n, w_next=w)
    n = n.cpu()
    assert (n[0] == 0).all() and torch.isnan(n[2]).all() and torch.isnan(n[3, 9])
    ref, _ = norm_ref(x[[1, 4, 5]].double().cpu(), w.cpu())
    check("n", n[[1, 4, 5]], ref, (r_tol(d) + 3 * U) * ref.abs() + half_step(ref, torch.float32))


def grad_ref(s, y, rp, rn, alpha, has=("dy", "dn", "b", "post")):
    """The gradients by the formulas, and the magnitudes that rounding scales with."""
    wn, d = s["w_next"].double(), y.shape[1]
    dx = s["dy"].double() if "dy" in has else torch.zeros(y.shape, dtype=torch.float64)
    mag = dx.abs()
    out = {}
    if "dn" in has:
        u, h = y * rn, s["dn"].double() * wn
        dx = dx + rn * (h - u * (h * u).mean(1, keepdim=True))
        mag = mag + rn * (h.abs() + u.abs() * (h * u).abs().mean(1, keepdim=True))
        out["dw_next"] = ((s["dn"].double() * u).sum(0), (s["dn"].double() * u).abs().sum(0))
    out["dx"] = (dx, mag)
    if "b" in has:
        g = col(s["gate"])
        w = s["w_post"].double() if "post" in has else torch.ones(d, dtype=torch.float64)
        c = s["b"].double() * (rp if "post" in has else 1.0)
        e, em = alpha * g * dx, abs(alpha) * (g if s["gate"] is not None else 1.0) * mag
        if "post" in has:
            h, hm = w * e, w.abs() * em
            db = rp * (h - c * (h * c).mean(1, keepdim=True))
            out["db"] = (db, rp * (hm + c.abs() * (hm * c.abs()).mean(1, keepdim=True)))
            out["dw_post"] = ((e * c).sum(0), (em * c.abs()).sum(0))
        else:
            out["db"] = (e, em)
        if s["gate"] is not None:
            dg, dgm = alpha * dx * c * w, abs(alpha) * mag * (c * w).abs()
            out["dgate"] = (dg, dgm) if s["gate"].dim() == 2 else (dg.sum(1), dgm.sum(1))
    return out


@pytest.mark.parametrize("T,d", SIZES + [(2500, 64), (1100, 2048)])
@pytest.mark.parametrize("types,gate", list(itertools.product(TYPES[:4], ["none", "token", "full"])))
def test_gradients(T, d, types, gate):
    sdt, adt, wdt = types
    print(f"[case] norm gradient {T} {d} {types} {gate}", flush=True)
    s = inputs(T, d, sdt, adt, wdt, gate, seed=4)
    c = {k: (v.cuda() if v is not None else None) for k, v in s.items()}
    y, n = torch.empty_like(c["x"]), torch.empty_like(c["b"])
    rp, rn = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    tq.norm_residual(c["x"], y=y, n=n, b=c["b"], w_post=c["w_post"], w_next=c["w_next"], gate=c["gate"],
                     alpha=0.75, rstd_post=rp, rstd_next=rn)
    o = dict(dx=torch.empty_like(c["x"]), db=torch.empty_like(c["b"]), dw_post=torch.empty(d, device="cuda"),
             dw_next=torch.empty(d, device="cuda"))
    if gate != "none":
        o["dgate"] = torch.empty_like(c["gate"])
    tq.norm_residual_grad(y, dy=c["dy"], dn=c["dn"], b=c["b"], w_post=c["w_post"], w_next=c["w_next"],
                          gate=c["gate"], alpha=0.75, rstd_post=rp, rstd_next=rn, **o)
    ref = grad_ref(s, y.double().cpu(), rp.double().cpu()[:, None], rn.double().cpu()[:, None], 0.75)
    for name, t in o.items():
        r, mag = ref[name]
        # a mean over the row (d U), the sums over rows (T U) or over the row
        # again, and at most 12 roundings of single values on the way
        check(name, t, r, (2 * d + T + 12) * U * mag + half_step(r, t.dtype))
    # the same inputs give the same bits
    again = {k: torch.empty_like(v) for k, v in o.items()}
    tq.norm_residual_grad(y, dy=c["dy"], dn=c["dn"], b=c["b"], w_post=c["w_post"], w_next=c["w_next"],
                          gate=c["gate"], alpha=0.75, rstd_post=rp, rstd_next=rn, **again)
    assert all(torch.equal(o[k], again[k]) for k in o)


@pytest.mark.parametrize("has", [("dn",), ("dy", "b"), ("dy", "b", "post"), ("dn", "b"), ("dn", "b", "post")])
def test_parts_of_the_gradients(has):
    T, d = 21, 392
    s = inputs(T, d, "f32", "f16", "f32", "token" if "b" in has else "none", seed=5)
    c = {k: (v.cuda() if v is not None else None) for k, v in s.items()}
    y, rn = c["x"], torch.empty(T, device="cuda")
    tq.norm_residual(y, n=torch.empty_like(c["b"]), w_next=c["w_next"], rstd_next=rn)
    rp = (c["b"].double().pow(2).mean(1) + EPS).rsqrt().float()
    o, kw = dict(dx=torch.empty_like(c["x"])), {}
    if "dy" in has:
        kw["dy"] = c["dy"]
    if "dn" in has:
        kw.update(dn=c["dn"], w_next=c["w_next"], rstd_next=rn)
        o["dw_next"] = torch.empty(d, device="cuda")
    if "b" in has:
        kw.update(b=c["b"], gate=c["gate"])
        o["db"], o["dgate"] = torch.empty_like(c["b"]), torch.empty_like(c["gate"])
    if "post" in has:
        kw.update(w_post=c["w_post"], rstd_post=rp)
        o["dw_post"] = torch.empty(d, device="cuda")
    tq.norm_residual_grad(y, alpha=1.5, **kw, **o)
    ref = grad_ref(s, y.double().cpu(), rp.double().cpu()[:, None], rn.double().cpu()[:, None], 1.5, has)
    for name, t in o.items():
        r, mag = ref[name]
        check(name, t, r, (2 * d + T + 12) * U * mag + half_step(r, t.dtype))
    # each output alone, and in place of an input
    for name in o:
        one = {name: torch.full_like(o[name], 3.0)}
        tq.norm_residual_grad(y, alpha=1.5, **kw, **one)
        assert torch.equal(one[name], o[name]), name
    if "dy" in has:
        t = c["dy"].clone()
        tq.norm_residual_grad(y, alpha=1.5, **{**kw, "dy": t}, dx=t)
        assert torch.equal(t, o["dx"])
    if "dn" in has and "b" in has:
        t = c["dn"].clone()
        tq.norm_residual_grad(y, alpha=1.5, **{**kw, "dn": t}, db=t)
        assert torch.equal(t, o["db"])


def test_gradients_against_differences():
    """The derivative of sum(dy y + dn n) along a direction, by the formulas in
    64 bits at +-h, is the gradients' product with it: off by O(h^2) and by the
    gradients' own f32 rounding."""
    T, d, h, alpha = 4, 136, 1e-4, 0.75
    s = inputs(T, d, "f32", "f32", "f32", "token", seed=6)
    c = {k: v.cuda() for k, v in s.items()}
    y, n = torch.empty_like(c["x"]), torch.empty_like(c["b"])
    rp, rn = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    tq.norm_residual(c["x"], y=y, n=n, b=c["b"], w_post=c["w_post"], w_next=c["w_next"], gate=c["gate"],
                     alpha=alpha, rstd_post=rp, rstd_next=rn)
    o = dict(dx=torch.empty_like(y), db=torch.empty_like(n), dw_post=torch.empty(d, device="cuda"),
             dw_next=torch.empty(d, device="cuda"), dgate=torch.empty(T, device="cuda"))
    tq.norm_residual_grad(y, dy=c["dy"], dn=c["dn"], b=c["b"], w_post=c["w_post"], w_next=c["w_next"],
                          gate=c["gate"], alpha=alpha, rstd_post=rp, rstd_next=rn, **o)
    for k, grad in (("x", "dx"), ("b", "db"), ("w_post", "dw_post"), ("w_next", "dw_next"), ("gate", "dgate")):
        v = torch.randn(s[k].shape, generator=gen(7), dtype=torch.float64)

        def loss(t):
            q = dict(s)
            q[k] = s[k].double() + t * v
            yy, _, _ = forward_ref(q, alpha)
            nn, _ = norm_ref(yy, q["w_next"])
            return float((s["dy"].double() * yy + s["dn"].double() * nn).sum())

        num = (loss(h) - loss(-h)) / (2 * h)
        prod = o[grad].double().cpu() * v
        # third derivatives of the norms are below 100 / rms^3 here (rms > 0.5):
        # h^2 / 6 * 800 per value; f32 rounding as in test_gradients
        tol = h * h / 6 * 800 * T * d + (2 * d + T + 12) * U * 20 * float(prod.abs().sum())
        assert abs(num - float(prod.sum())) <= tol, (k, num, float(prod.sum()), tol)


def test_no_rows():
    d = 64
    x = torch.empty((0, d), device="cuda")
    tq.norm_residual(x, n=x, w_next=torch.ones(d, device="cuda"))
    dw = torch.full((d,), 4.0, device="cuda")
    r = torch.empty(0, device="cuda")
    tq.norm_residual_grad(x, dx=x, dy=x, dn=x, w_next=torch.ones(d, device="cuda"), rstd_next=r, dw_next=dw)
    assert (dw == 0).all()


def test_graph_replay_stream_and_workspace():
    T, d = 600, 1032
    s = inputs(T, d, "bf16", "bf16", "bf16", "token", seed=8)
    c = {k: v.cuda() for k, v in s.items()}
    y, n = torch.empty_like(c["x"]), torch.empty_like(c["b"])
    rp, rn = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    o = dict(dx=torch.empty_like(c["x"]), db=torch.empty_like(c["b"]), dw_post=torch.empty(d, device="cuda"),
             dw_next=torch.empty(d, device="cuda"), dgate=torch.empty(T, device="cuda"))
    ws = torch.full((ops.norm_grad_workspace(T, d),), 255, dtype=torch.uint8, device="cuda")

    def step(stream=None):
        tq.norm_residual(c["x"], y=y, n=n, b=c["b"], w_post=c["w_post"], w_next=c["w_next"], gate=c["gate"],
                         alpha=0.75, rstd_post=rp, rstd_next=rn, stream=stream)
        tq.norm_residual_grad(y, dy=c["dy"], dn=c["dn"], b=c["b"], w_post=c["w_post"], w_next=c["w_next"],
                              gate=c["gate"], alpha=0.75, rstd_post=rp, rstd_next=rn, ws=ws, stream=stream, **o)

    step()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in o.items()}
    side = torch.cuda.Stream()
    for k, v in o.items():
        v.fill_(float("nan"))
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    assert all(torch.equal(o[k], want[k]) for k in o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for v in o.values():
            v.fill_(float("nan"))
        ws.fill_(255)
        torch.randn(1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], want[k]) for k in o)
