"""Products grouped by expert against plain sums in 64 bits: ragged, empty and
single-row groups, odd sizes, gathered rows, strides, rows outside every group,
not-a-number in rows that must not be read, malformed offsets, graphs, streams."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import DT, check, gen, half_step, normal, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# name, row counts, d_in, d_out: every tile shape, with group edges inside and
# outside tiles
SHAPES = [
    ("one row", [1], 128, 64),
    ("single rows", [1, 0, 1, 1, 0, 1], 8, 16),
    ("decode", [3, 0, 16, 1, 17, 5], 264, 136),
    ("decode wide", [2, 1], 2048, 1408),
    ("small odd", [33, 64, 0, 31], 72, 200),
    ("middle", [129, 0, 128, 300, 1], 328, 264),
    ("middle empty ends", [0, 0, 200, 150, 0], 64, 128),
    ("long", [1030, 515], 520, 1032),
    ("one group", [777], 136, 392),
    ("hot", [2000, 3, 0, 1, 60], 256, 520),
    ("long k", [70, 40], 4104, 72),
    ("large tiles", [4096 + 5], 192, 4096 + 8),
]


def make(counts, d_in, d_out, dt, seed, gather=0, lead=0, tail=0, wide=0):
    """Rows before the first and after the last group hold NaN; with `wide`,
    the columns after a row do too."""
    g = gen(seed)
    off = offsets(counts, lead)
    rows = off[-1] + tail
    x_rows = rows if not gather else max(1, rows // gather)
    nan = float("nan")
    x = torch.full((x_rows, d_in + wide), nan, dtype=dt)
    x[:, :d_in] = normal(g, (x_rows, d_in), 1.0, dt)
    dy = torch.full((rows, d_out + wide), nan, dtype=dt)
    dy[:, :d_out] = normal(g, (rows, d_out), 1.0, dt)
    src = None
    if gather:
        src = torch.randint(0, x_rows * gather, (rows,), generator=g, dtype=torch.int32)
    else:
        x[:lead], x[off[-1]:] = nan, nan
    dy[:lead], dy[off[-1]:] = nan, nan
    w = normal(g, (len(counts), d_out, d_in), 1.0, dt)
    return off, rows, x, dy, w, src


def dev(t):
    return None if t is None else t.cuda()


def source(x, src, div, d_in, rows):
    x = x[:, :d_in].double()
    return x if src is None else x[(src.long() // div)]


@pytest.mark.parametrize("name,counts,d_in,d_out", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["plain", "gather", "strided"])
def test_forward(name, counts, d_in, d_out, dtype, kind):
    print(f"[case] forward {name} {dtype} {kind}", flush=True)
    dt, out = DT[dtype], {"plain": DT[dtype], "gather": torch.float32, "strided": torch.bfloat16}[kind]
    gather, wide = (3 if kind == "gather" else 0), (8 if kind == "strided" else 0)
    off, rows, x, dy, w, src = make(counts, d_in, d_out, dt, 1, gather, lead=2, tail=3, wide=wide)
    full = torch.full((rows, d_out + wide), -7.0, dtype=out, device="cuda")
    xd = x.cuda()
    tq.group_gemm(xd[:, :d_in], w.cuda(), full[:, :d_out],
                  off=torch.tensor(off, dtype=torch.int32, device="cuda"), src=dev(src), src_div=max(gather, 1))
    torch.cuda.synchronize()
    xs = source(x, src, gather, d_in, rows)
    got = full.cpu()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        a, b = xs[lo:hi], w[e].double()
        ref, mag = a @ b.t(), a.abs() @ b.abs().t()
        check(f"expert {e}", got[lo:hi, :d_out], ref, d_in * 2.0 ** -23 * mag + half_step(ref, out))
    assert (got[:off[0]] == -7).all() and (got[off[-1]:] == -7).all(), "rows outside the groups were written"
    assert (got[:, d_out:] == -7).all(), "columns after the rows were written"


@pytest.mark.parametrize("name,counts,d_in,d_out", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["plain", "strided"])
def test_input_gradient(name, counts, d_in, d_out, dtype, kind):
    print(f"[case] dx {name} {dtype} {kind}", flush=True)
    dt, out = DT[dtype], DT[dtype] if kind == "plain" else torch.float32
    wide = 8 if kind == "strided" else 0
    off, rows, x, dy, w, _ = make(counts, d_in, d_out, dt, 2, 0, lead=1, tail=2, wide=wide)
    full = torch.full((rows, d_in + wide), -7.0, dtype=out, device="cuda")
    dyd = dy.cuda()
    tq.group_gemm_dx(dyd[:, :d_out], w.cuda(), full[:, :d_in],
                     off=torch.tensor(off, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    got, dys = full.cpu(), dy[:, :d_out].double()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        a, b = dys[lo:hi], w[e].double()
        ref, mag = a @ b, a.abs() @ b.abs()
        check(f"expert {e}", got[lo:hi, :d_in], ref, d_out * 2.0 ** -23 * mag + half_step(ref, out))
    assert (got[:off[0]] == -7).all() and (got[off[-1]:] == -7).all(), "rows outside the groups were written"
    assert (got[:, d_in:] == -7).all(), "columns after the rows were written"


@pytest.mark.parametrize("name,counts,d_in,d_out", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["plain", "gather", "strided"])
def test_weight_gradient(name, counts, d_in, d_out, dtype, kind):
    print(f"[case] dw {name} {dtype} {kind}", flush=True)
    dt, out = DT[dtype], torch.float32 if kind == "plain" else DT[dtype]
    gather, wide = (2 if kind == "gather" else 0), (8 if kind == "strided" else 0)
    off, rows, x, dy, w, src = make(counts, d_in, d_out, dt, 3, gather, lead=1, tail=2, wide=wide)
    dw = torch.full((len(counts), d_out, d_in), -7.0, dtype=out, device="cuda")
    xd, dyd = x.cuda(), dy.cuda()
    tq.group_gemm_dw(dyd[:, :d_out], xd[:, :d_in], dw, off=torch.tensor(off, dtype=torch.int32, device="cuda"),
                     src=dev(src), src_div=max(gather, 1))
    torch.cuda.synchronize()
    xs, dys = source(x, src, gather, d_in, rows), dy[:, :d_out].double()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        a, b = dys[lo:hi].t(), xs[lo:hi]
        ref, mag = a @ b, a.abs() @ b.abs()
        check(f"expert {e}", dw[e], ref, (hi - lo) * 2.0 ** -23 * mag + half_step(ref, out))


def test_gradients_are_those_of_the_product():
    """<dy, y(x + h v)> - <dy, y(x - h v)> over 2h is <dx, v>, and the same for w:
    y is linear in each, so the difference is exact up to rounding."""
    counts, d_in, d_out = [5, 0, 40], 96, 72
    off, rows, x, dy, w, _ = make(counts, d_in, d_out, torch.float16, 4)
    offd = torch.tensor(off, dtype=torch.int32, device="cuda")
    v, u = normal(gen(5), x.shape, 1.0, torch.float16), normal(gen(6), w.shape, 1.0, torch.float16)

    def loss(a, b):
        y = torch.zeros((rows, d_out), device="cuda")
        tq.group_gemm(a.cuda(), b.cuda(), y, off=offd)
        return float((y.double().cpu() * dy.double()).sum())

    dx, dw = torch.zeros((rows, d_in), device="cuda"), torch.zeros(w.shape, device="cuda")
    tq.group_gemm_dx(dy.cuda(), w.cuda(), dx, off=offd)
    tq.group_gemm_dw(dy.cuda(), x.cuda(), dw, off=offd)
    # steps of x and w that 16 bits hold exactly
    xp, wp = (x + v).half(), (w + u).half()
    for got, plus, base, grad in ((loss(xp, w), loss(x, w), (xp.double() - x.double()), dx),
                                  (loss(x, wp), loss(x, w), (wp.double() - w.double()), dw)):
        want = float((grad.double().cpu() * base).sum())
        # every y is off by at most d_in 2^-23 of the sum of its magnitudes
        mag = sum(float((dy[lo:hi].double().abs() @ (w[e].double().abs() + u[e].double().abs())
                         * (x[lo:hi].double().abs() + v[lo:hi].double().abs())).sum())
                  for e, (lo, hi) in enumerate(zip(off, off[1:])))
        assert abs(got - plus - want) <= 2 * (d_in + d_out + rows) * 2.0 ** -23 * mag


def test_index_outside_x_reads_as_zero():
    x, w = torch.ones((4, 64), dtype=torch.float16, device="cuda"), torch.ones((2, 32, 64), dtype=torch.float16, device="cuda")
    src = torch.tensor([0, -1, 3, 4, 2 ** 31 - 1, 1, -2 ** 31, 2], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 5, 8], dtype=torch.int32, device="cuda")
    y = torch.full((8, 32), -7.0, device="cuda")
    tq.group_gemm(x, w, y, off=off, src=src)
    want = torch.tensor([64.0, 0, 64, 0, 0, 64, 0, 64])
    assert torch.equal(y.cpu(), want[:, None].expand(8, 32))
    dw = torch.full((2, 32, 64), -7.0, device="cuda")
    tq.group_gemm_dw(torch.ones((8, 32), dtype=torch.float16, device="cuda"), x, dw, off=off, src=src)
    assert (dw[0] == 2).all() and (dw[1] == 2).all()


@pytest.mark.parametrize("div", [1, 2, 3, 4, 6, 7, 8, 1000])
def test_source_index_division(div):
    """src / src_div for every remainder, at the largest indices too."""
    x_rows = 64
    x = torch.zeros((x_rows, 64), dtype=torch.float16, device="cuda")
    x[:, 0] = torch.arange(x_rows, device="cuda").half()
    src = torch.arange(0, x_rows * div, dtype=torch.int32, device="cuda")[-4096:].contiguous()
    w = torch.zeros((1, 16, 64), dtype=torch.float16, device="cuda")
    w[0, :, 0] = 1
    y = torch.empty((len(src), 16), device="cuda")
    tq.group_gemm(x, w, y, src=src, src_div=div)
    assert torch.equal(y[:, 0].cpu(), (src.cpu() // div).float())


@pytest.mark.parametrize("off", [[-5, 3, 40, 40], [0, 100, 7, 64], [64, 0, 0, 0], [9, 9, 9, 9],
                                 [2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1]])
def test_any_offsets_stay_inside(off):
    """Offsets that break the rules give unspecified results, inside the arrays."""
    rows, d = 64, 64
    big = torch.full((3 * rows, d), -7.0, dtype=torch.float16, device="cuda")
    x, y = torch.ones((rows, d), dtype=torch.float16, device="cuda"), big[rows:2 * rows]
    w = torch.ones((3, d, d), dtype=torch.float16, device="cuda")
    offd = torch.tensor(off, dtype=torch.int32, device="cuda")
    tq.group_gemm(x, w, y, off=offd)
    tq.group_gemm_dx(x, w, y, off=offd)
    dw = torch.full((5, d, d), -7.0, dtype=torch.float16, device="cuda")
    tq.group_gemm_dw(x, x, dw[1:4], off=offd)
    torch.cuda.synchronize()
    assert (big[:rows] == -7).all() and (big[2 * rows:] == -7).all()
    assert (dw[0] == -7).all() and (dw[4] == -7).all()


def test_no_rows():
    w = torch.ones((2, 32, 64), dtype=torch.bfloat16, device="cuda")
    x, y = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 32), device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    tq.group_gemm(x, w, y, off=off)
    tq.group_gemm_dx(y.to(torch.bfloat16), w, x, off=off)
    dw = torch.full((2, 32, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    tq.group_gemm_dw(y.to(torch.bfloat16), x, dw, off=off)
    assert (dw == 0).all()


def test_special_values_stay_in_their_rows():
    """An infinity or NaN of one row reaches that row's outputs alone."""
    x = torch.ones((40, 72), dtype=torch.float16)
    x[7, 3], x[20, 71] = float("inf"), float("nan")
    w = torch.ones((2, 24, 72), dtype=torch.float16, device="cuda")
    off = torch.tensor([0, 19, 40], dtype=torch.int32, device="cuda")
    y = torch.empty((40, 24), device="cuda")
    tq.group_gemm(x.cuda(), w, y, off=off)
    y = y.cpu()
    assert torch.isinf(y[7]).all() and torch.isnan(y[20]).all()
    keep = [r for r in range(40) if r not in (7, 20)]
    assert (y[keep] == 72).all()
    # ... and an expert's weight gradient does not see the rows of another
    dw = torch.empty((2, 24, 72), device="cuda")
    tq.group_gemm_dw(torch.ones((40, 24), dtype=torch.float16, device="cuda"), x.cuda(), dw, off=off)
    assert torch.isfinite(dw[1, :, :71]).all() and torch.isnan(dw[1, :, 71]).all()
    assert torch.isinf(dw[0, :, 3]).all() and (dw[0, :, 4:] == 19).all()


def test_many_groups():
    """More groups than a wave has lanes, most of them empty."""
    G, d = 1000, 64
    counts = [(i * 7 % 11 == 0) * (i % 5) for i in range(G)]
    off, rows, x, dy, w, _ = make(counts, d, d, torch.bfloat16, 8)
    y = torch.empty((rows, d), device="cuda")
    offd = torch.tensor(off, dtype=torch.int32, device="cuda")
    tq.group_gemm(x.cuda(), w.cuda(), y, off=offd)
    grp = torch.repeat_interleave(torch.arange(G), torch.tensor(counts))
    ref = (x.double()[:, None, :] @ w.double()[grp].transpose(1, 2))[:, 0]
    mag = (x.double().abs()[:, None, :] @ w.double().abs()[grp].transpose(1, 2))[:, 0]
    check("y", y, ref, d * 2.0 ** -23 * mag + half_step(ref, torch.float32))


def test_graph_replay_and_another_stream():
    counts, d_in, d_out = [100, 0, 37, 300], 256, 192
    off, rows, x, dy, w, _ = make(counts, d_in, d_out, torch.bfloat16, 9)
    x, dy, w = x.cuda(), dy.cuda(), w.cuda()
    offd = torch.tensor(off, dtype=torch.int32, device="cuda")
    y, dx = torch.empty((rows, d_out), device="cuda"), torch.empty((rows, d_in), device="cuda")
    dw = torch.empty(w.shape, device="cuda")

    def step(stream=None):
        tq.group_gemm(x, w, y, off=offd, stream=stream)
        tq.group_gemm_dx(dy, w, dx, off=offd, stream=stream)
        tq.group_gemm_dw(dy, x, dw, off=offd, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, dw)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in (y, dx, dw):
        t.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (y, dx, dw):
            t.fill_(float("nan"))
        torch.randn(1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), want))


def test_rows_past_32_bit_offsets():
    """x and y of more than 2^32 bytes: the last rows are as right as the first."""
    rows, d = (1 << 21) + 300, 1032
    x = torch.zeros((rows, d), dtype=torch.float16, device="cuda")
    x[:300], x[-300:] = 1.0, 2.0
    w = torch.ones((2, 16, d), dtype=torch.float16, device="cuda")
    y = torch.empty((rows, 16), device="cuda")
    off = torch.tensor([0, rows - 200, rows], dtype=torch.int32, device="cuda")
    tq.group_gemm(x, w, y, off=off)
    assert (y[:300] == d).all() and (y[-300:] == 2 * d).all() and (y[300:-300] == 0).all()
    dx = torch.empty((rows, d), dtype=torch.float16, device="cuda")
    tq.group_gemm_dx(y[:, :8].half().contiguous(), w[:, :8].contiguous(), dx, off=off)
    assert (dx[:300] == 8 * d).all() and (dx[-300:] == 16 * d).all() and (dx[300:-300] == 0).all()
    dw = torch.empty((2, 8, d), device="cuda")
    tq.group_gemm_dw(torch.ones((rows, 8), dtype=torch.float16, device="cuda"), x, dw, off=off)
    assert (dw[0] == 300 + 200).all() and (dw[1] == 400).all()


def test_offsets_that_count_too_many_tiles():
    """Offsets that give every group all rows (so that tiles are counted again
    and again): still no access outside the arrays."""
    G, rows, d = 1000, 4096, 64
    big = torch.full((3 * rows, d), -7.0, dtype=torch.float16, device="cuda")
    x, y = torch.ones((rows, d), dtype=torch.float16, device="cuda"), big[rows:2 * rows]
    w = torch.ones((G, d, d), dtype=torch.float16, device="cuda")
    off = torch.tensor([0, rows] * (G // 2) + [0], dtype=torch.int32, device="cuda")
    for g, o in ((G, off), (64, off[:65].contiguous())):
        tq.group_gemm(x, w[:g], y, off=o)
        tq.group_gemm_dx(x, w[:g], y, off=o)
    torch.cuda.synchronize()
    assert (big[:rows] == -7).all() and (big[2 * rows:] == -7).all()


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("dtype,value", [("f16", 2.0 ** -20), ("f16", 2.0 ** -24), ("bf16", 2.0 ** -128), ("bf16", 2.0 ** -132)])
def test_subnormal_values_count(rows, dtype, value):
    """Values below the smallest normal are not lost: sums of powers of two, exact."""
    dt, d, o = DT[dtype], 64, 16
    x = torch.full((rows, d), value, dtype=dt, device="cuda")
    w, one = torch.ones((1, o, d), dtype=dt, device="cuda"), torch.ones((rows, o), dtype=dt, device="cuda")
    y, dx, dw = (torch.empty(s, device="cuda") for s in ((rows, o), (rows, d), (1, o, d)))
    tq.group_gemm(x, w, y)
    tq.group_gemm_dx(one * value, w, dx)
    tq.group_gemm_dw(one, x, dw)
    assert (y.double() == d * value).all() and (dx.double() == o * value).all()
    # a sum of `rows` equal terms of one bit: exact in f32
    assert (dw.double() == rows * value).all()


@pytest.mark.parametrize("G", [63, 64, 65, 130])
def test_gradients_of_many_groups(G):
    """Around and above the groups that a wave holds at once, a few of them heavy."""
    d_in, d_out = 72, 136
    counts = [(i * 5 % 7 == 0) * (i % 4) + 150 * (i in (3, G - 1)) for i in range(G)]
    off, rows, x, dy, w, _ = make(counts, d_in, d_out, torch.float16, 10)
    offd = torch.tensor(off, dtype=torch.int32, device="cuda")
    dx, dw = torch.empty((rows, d_in), device="cuda"), torch.empty((G, d_out, d_in), device="cuda")
    tq.group_gemm_dx(dy.cuda(), w.cuda(), dx, off=offd)
    tq.group_gemm_dw(dy.cuda(), x.cuda(), dw, off=offd)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        a, b, c = dy[lo:hi].double(), w[e].double(), x[lo:hi].double()
        check(f"dx {e}", dx[lo:hi], a @ b, d_out * 2.0 ** -23 * (a.abs() @ b.abs()) + half_step(a @ b, torch.float32))
        ref = a.t() @ c
        check(f"dw {e}", dw[e], ref, (hi - lo) * 2.0 ** -23 * (a.t().abs() @ c.abs()) + half_step(ref, torch.float32))
