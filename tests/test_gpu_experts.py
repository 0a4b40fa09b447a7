"""A whole layer of experts for a few tokens, against the formula in 64 bits.

Bounds.  a = W x sums d products exact in f32 (16-bit values, or 8-bit integers
times 16-bit values): d 2^-23 of the sum of magnitudes A; 8-bit weights: one
rounding more for the scale.  silu has a slope below 1.1 and is no larger than
its argument, its f32 value is within 2^-20 (|g| 2^-24 of the exponential's
argument, |g| < 8 here where it counts, and some ulps): h before rounding is off
by 1.1 eA_g |u| + |g| eA_u + 2^-20 |h|, and by half a step after it.  y sums ff k
products: (ff + k + 4) 2^-23 of the magnitudes, and what comes of h's error."""
import numpy as np
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.int8_cases import quantised
from tests.ops_util import DT, check, gen, half_step, normal

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def make(E, T, k, d, ff, dtype, int8, seed, repeat=False, bad=False):
    g = gen(seed)
    dt = DT[dtype]
    x = normal(g, (T, d), 1.0, dt)
    if repeat:
        ids = torch.randint(0, E, (T, k), generator=g)
    else:
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    ids = ids.to(I32)
    if bad:
        r = torch.rand((T, k), generator=g)
        ids[r < 0.25] = -1
        ids[r > 0.9] = E
    w = torch.softmax(torch.randn((T, k), generator=g), 1)
    w_up, w_down = normal(g, (E, 2 * ff, d), d ** -0.5, dt), normal(g, (E, d, ff), ff ** -0.5, dt)
    s_up = s_down = None
    if int8:
        w_up, s_up = quantised(w_up.view(-1, d))
        w_down, s_down = quantised(w_down.view(-1, ff))
        w_up, s_up = w_up.view(E, 2 * ff, d), s_up.view(E, 2 * ff)
        w_down, s_down = w_down.view(E, d, ff), s_down.view(E, d)
    return x, ids, w, w_up, w_down, s_up, s_down


def reference(x, ids, w, w_up, w_down, s_up, s_down, dt):
    """y without add in 64 bits, and the bound before the last rounding."""
    E, d, ff = w_down.shape
    T, k = ids.shape
    y, tol = torch.zeros((T, d), dtype=torch.float64), torch.zeros((T, d), dtype=torch.float64)
    xd = x.double()
    eps = 2.0 ** -23
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        u, v = w_up[e].double(), w_down[e].double()
        if s_up is not None:
            u, v = u * s_up[e].double()[:, None], v * s_down[e].double()[:, None]
        a, A = xd[t] @ u.t(), xd[t].abs() @ u.abs().t()
        ea = (d + 1) * eps * A
        (g, up), (eg, eu) = a.chunk(2, 1), ea.chunk(2, 1)
        h = g * torch.sigmoid(g) * up
        eh = 1.1 * eg * up.abs() + g.abs() * eu + 1.1 * eg * eu + 2.0 ** -20 * h.abs()
        eh = eh + half_step(h.abs() + eh, dt)
        h = h.to(dt).double()
        # (the rounded reference and the rounded result may lie a step apart)
        eh = eh + half_step(h, dt)
        z, Z = h @ v.t(), h.abs() @ v.abs().t()
        c = w[t, j].double()[:, None]
        y.index_add_(0, t, c * z)
        tol.index_add_(0, t, c.abs() * ((ff + k + 4) * eps * Z + eh @ v.abs().t()))
    return y, tol


def run(m, ydt="f32", add=None, T=None, ws=None, **kw):
    x, ids, w, w_up, w_down, s_up, s_down = [None if t is None else t.cuda() for t in m]
    y = torch.full((x.shape[0], w_down.shape[1]), -7.0, dtype=DT[ydt], device="cuda")
    if ws is None:
        n = tq.experts_workspace(ids.shape[0], ids.shape[1], w_down.shape[0], w_down.shape[1], w_down.shape[2])
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    tq.experts_forward(x, ids, w, w_up, w_down, y, ws, s_up=s_up, s_down=s_down, add=add, **kw)
    return y


# experts, tokens, topk, d, ff: slots below, at and above the experts; 1, 16, 17, 33 and
# more slots of one expert; sizes that end inside a fragment, a step, a run
SIZES = [(8, 1, 1, 64, 48), (8, 1, 2, 256, 96), (60, 1, 4, 256, 136), (60, 5, 4, 520, 264), (60, 32, 4, 256, 96),
         (8, 16, 2, 136, 72), (8, 17, 2, 256, 136), (8, 40, 2, 136, 264), (3, 64, 2, 264, 72), (1, 33, 1, 64, 40),
         (1, 100, 1, 128, 64), (2, 512, 2, 64, 32), (128, 3, 8, 72, 24), (1024, 2, 32, 16, 16), (300, 128, 8, 32, 16),
         (4, 2, 2, 4096, 2056), (2, 1, 1, 1032, 5000), (5, 1, 3, 4104, 200), (40, 1, 32, 48, 24), (6, 1, 2, 2048, 1032)]


@pytest.mark.parametrize("E,T,k,d,ff", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("int8", [False, True])
def test_layer(E, T, k, d, ff, dtype, int8):
    if int8:
        d, ff = -(-d // 16) * 16, -(-ff // 16) * 16
    print(f"[case] layer {E} {T} {k} {d} {ff} {dtype} {int8}", flush=True)
    m = make(E, T, k, d, ff, dtype, int8, 1)
    y = run(m)
    ref, tol = reference(*m, DT[dtype])
    check("y", y, ref, 1.01 * tol + half_step(ref, torch.float32))
    # rounded to 16 bits: the same values
    for ydt in ("f16", "bf16"):
        assert torch.equal(run(m, ydt), y.to(DT[ydt]))


@pytest.mark.parametrize("E,T,k,d,ff", [(8, 6, 3, 128, 80), (2, 30, 2, 128, 80), (40, 4, 4, 128, 80), (1, 20, 4, 64, 48),
                                        (3, 1, 8, 128, 80), (12, 1, 5, 4112, 336)])
@pytest.mark.parametrize("int8", [False, True])
def test_an_expert_named_twice_and_ids_outside(E, T, k, d, ff, int8):
    for repeat, bad in ((True, False), (False, True), (True, True)):
        if not repeat and k > E:
            continue
        m = make(E, T, k, d, ff, "bf16", int8, 2, repeat, bad)
        print(f"[case] layer ids {E} {T} {k} {repeat} {bad} {int8}", flush=True)
        add = normal(gen(3), (T, d), 1.0, torch.float32)
        y = run(m, add=add.cuda())
        m[2][(m[1] < 0) | (m[1] >= E)] = 0.0
        ref, tol = reference(*m, torch.bfloat16)
        ref = ref + add.double()
        check("y", y, ref, 1.01 * tol + 2 * half_step(ref, torch.float32) + 2.0 ** -24 * add.double().abs())


@pytest.mark.parametrize("E,T", [(8, 1), (8, 2), (2, 30)])
def test_no_slot_counts(E, T):
    m = make(E, T, 2, 64, 48, "f16", False, 4)
    m[1][:] = torch.tensor([-1, E], dtype=I32)
    m[2][:] = float("nan")
    assert (run(m) == 0).all()
    add = torch.randn((T, 64), device="cuda", dtype=torch.float16)
    assert torch.equal(run(m, "f16", add=add), add)


def test_strides_residual_in_place_and_neighbours():
    E, T, k, d, ff = 8, 9, 2, 136, 72
    m = list(make(E, T, k, d, ff, "f16", False, 5))
    wide = torch.full((T, d + 24), float("nan"), dtype=torch.float16)
    wide[:, :d] = m[0]
    y = torch.full((T, d + 5), -7.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(tq.experts_workspace(T, k, E, d, ff), dtype=torch.uint8, device="cuda")
    c = [t.cuda() for t in m[1:5]]
    add = normal(gen(6), (T, d + 3), 1.0, torch.float16).cuda()
    xw = wide.cuda()
    tq.experts_forward(xw[:, :d], *c, y[:, :d], ws, add=add[:, 1:d + 1])
    want = run(m, "f16", add=add[:, 1:d + 1].contiguous())
    assert torch.equal(y[:, :d], want) and (y[:, d:] == -7).all()
    # the residual stream: y is x, and add is x
    x = m[0].cuda()
    want = run(m, "f16", add=x)
    tq.experts_forward(x, *c, x, ws, add=x)
    assert torch.equal(x, want)


def test_the_same_bits_every_time_and_workspaces_in_turn():
    """The last workgroup differs from call to call, the sum does not; a
    workspace may hold anything, and serve calls of other sizes in between."""
    big, small = make(60, 24, 4, 512, 264, "bf16", False, 7), make(8, 3, 2, 128, 64, "bf16", True, 8)
    n = max(tq.experts_workspace(24, 4, 60, 512, 264), tq.experts_workspace(3, 2, 8, 128, 64))
    ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")
    b = [None if t is None else t.cuda() for t in big]
    s = [None if t is None else t.cuda() for t in small]
    yb, ys = torch.empty((24, 512), device="cuda"), torch.empty((3, 128), device="cuda")

    def both():
        tq.experts_forward(*b[:5], yb, ws)
        tq.experts_forward(*s[:5], ys, ws, s_up=s[5], s_down=s[6])

    both()
    wb, wsm = yb.clone(), ys.clone()
    for _ in range(30):
        yb.fill_(float("nan"))
        ys.fill_(float("nan"))
        both()
        assert torch.equal(yb, wb) and torch.equal(ys, wsm)


def test_graph_and_streams():
    m = make(16, 12, 3, 256, 136, "f16", False, 9)
    x, ids, w, w_up, w_down = [t.cuda() for t in m[:5]]
    y = torch.empty((12, 256), device="cuda")
    ws = torch.empty(tq.experts_workspace(12, 3, 16, 256, 136), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        tq.experts_forward(x, ids, w, w_up, w_down, y, ws, stream=stream)

    step()
    torch.cuda.synchronize()
    want = y.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for how in ("stream", "handle", "graph", "graph", "graph", "graph"):
        y.fill_(float("nan"))
        ws.fill_(255)
        torch.randn(1000, device="cuda").sum().item()
        torch.cuda.synchronize()
        if how == "graph":
            graph.replay()
        else:
            step(side if how == "stream" else side.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    # two calls at once, each with a workspace of its own
    y2, ws2, other = torch.empty_like(y), torch.empty_like(ws), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        tq.experts_forward(x, ids, w, w_up, w_down, y, ws, stream=side)
        tq.experts_forward(x, ids, w, w_up, w_down, y2, ws2, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(y2, want)
    # new ids and weights in a replayed graph
    m2 = make(16, 12, 3, 256, 136, "f16", False, 10)
    ids.copy_(m2[1])
    w.copy_(m2[2])
    graph.replay()
    torch.cuda.synchronize()
    new = y.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(y, new) and not torch.equal(new, want)


def test_no_tokens():
    m = make(4, 1, 2, 64, 32, "f16", False, 11)
    c = [t.cuda() for t in m[:5]]
    ws = torch.empty(tq.experts_workspace(0, 2, 4, 64, 32), dtype=torch.uint8, device="cuda")
    tq.experts_forward(c[0][:0], c[1][:0], c[2][:0], c[3], c[4], c[0][:0].clone(), ws)


def test_special_values_stay_with_their_tokens():
    E, T, k, d, ff = 4, 6, 2, 64, 48
    m = make(E, T, k, d, ff, "f16", False, 12)
    y = run(m)
    m[0][2, 5] = float("nan")
    m[0][4, 7] = float("inf")
    z = run(m)
    assert not torch.isfinite(z[2]).any() and not torch.isfinite(z[4]).any()
    keep = [0, 1, 3, 5]
    assert np.array_equal(z[keep].cpu().numpy(), y[keep].cpu().numpy())
