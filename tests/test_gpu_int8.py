"""8-bit integer products with a scale for each token and channel, and the
quantisation of their operands, against the definition: all values equal."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.group_cases import ragged
from tests.int8_cases import CASES, IDS, codes, kernel_of, product, quantised, ref_scale
from tests.ops_util import DT, gen, normal, offsets

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def same(a, b):
    """Equal values, not-a-number in the same places."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(3.5), b.nan_to_num(3.5))


# one wave a row below 2048 values, a workgroup above, read twice above 32768
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,d,wide", [(1, 16, 0), (5, 144, 8), (300, 1024, 0), (7, 1040, 16), (6, 2032, 8), (9, 2048, 8),
                                         (3, 2064, 0), (17, 4096, 0), (6, 4112, 8), (3, 8192, 0), (3, 8208, 8), (2, 14336, 0), (2, 32768, 0),
                                         (3, 32784, 8), (1, 131056, 0)])
def test_quant_rows(dtype, rows, d, wide):
    print(f"[case] int8 quant {dtype} {rows} {d} {wide}", flush=True)
    x = normal(gen(1), (rows, d + wide), 3.0, DT[dtype])
    x[0, :16] = 0
    if rows > 2:
        x[2] = 0
        x[1] *= 2.0 ** -12
    q = torch.full((rows, d), 77, dtype=torch.int8, device="cuda")
    c = torch.full((rows,), -7.0, device="cuda")
    tq.int8_quant_rows(x.cuda()[:, :d], q, c)
    rq, rc = quantised(x[:, :d])
    assert torch.equal(c.cpu(), rc)
    assert torch.equal(q.cpu(), rq)


def test_quant_weights():
    w = normal(gen(2), (3, 40, 272), 0.02, torch.bfloat16)
    q, c = torch.empty(w.shape, dtype=torch.int8, device="cuda"), torch.empty((3, 40), device="cuda")
    tq.int8_quant_rows(w.cuda(), q, c)
    rq, rc = quantised(w.view(120, 272))
    assert torch.equal(q.cpu().view(120, -1), rq) and torch.equal(c.cpu().view(-1), rc)


def test_quant_more_rows_than_workgroups():
    """65536 workgroups take rows in turns."""
    for rows, d in ((70000, 4112), (4 * 65536 + 70, 16)):
        x = torch.randn((rows, d), device="cuda", dtype=torch.float16)
        q, c = torch.empty((rows, d), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        tq.int8_quant_rows(x, q, c)
        for part in (slice(0, 300), slice(65400, 65700), slice(rows - 300, rows)):
            rq, rc = quantised(x[part].cpu())
            assert torch.equal(q[part].cpu(), rq) and torch.equal(c[part].cpu(), rc)


@pytest.mark.parametrize("d", [256, 5008])
def test_quant_special_values(d):
    x = torch.zeros((8, d))
    x[0] = 1e-45                          # below the smallest normal scale
    x[1] = torch.linspace(-3.0, 3.0, d) * 1e38
    x[2, 5] = float("inf")
    x[2, 6] = 1.0
    x[3, 200] = float("nan")
    x[3, 7] = 5.0
    x[4, :128] = 2.0 ** -149 * 127 * 1000
    x[5, 0], x[5, 1] = -0.0, -127.0
    x[6, 9] = float("-inf")
    x[7, :4] = torch.tensor([127.0, 0.5, -1.5, 2.5])        # ties to even
    q = torch.full((8, d), 77, dtype=torch.int8, device="cuda")
    c = torch.full((8,), -7.0, device="cuda")
    tq.int8_quant_rows(x.cuda(), q, c)
    rq, rc = quantised(x)
    assert torch.isnan(rc[[2, 3, 6]]).all() and (rq[[2, 3, 6]] == 0).all()
    assert rq[7, :4].tolist() == [127, 0, -2, 2]
    assert same(c.cpu(), rc) and torch.equal(q.cpu(), rq)
    h = torch.full((1, 16), 65504.0, dtype=torch.float16, device="cuda")
    tq.int8_quant_rows(h, q[:1, :16].contiguous(), c[:1])
    assert c[0].item() == ref_scale(torch.tensor(65504.0)).item()


def test_quotients_are_correctly_rounded():
    """Values next to the borders between codes, at scales from the smallest to
    the largest: equal to the definition, one by one."""
    g = gen(8)
    rows = []
    for e in (-126, -120, -100, -93, -92, -91, -60, -10, 0, 7, 60, 100, 120):
        amax = ((1 + torch.rand((64, 1), generator=g)) * 2.0 ** e * 127).clamp(max=3e38)
        c = ref_scale(amax)
        border = torch.randint(0, 127, (64, 256), generator=g).float() + 0.5
        x = (border.clamp(max=126.5) * c).to(torch.float32)
        x = (x.view(I32) + torch.randint(-2, 3, (64, 256), generator=g, dtype=I32)).clamp(min=0).view(torch.float32)
        x[:, 0] = amax[:, 0]
        rows.append(x * (torch.randint(0, 2, x.shape, generator=g) * 2 - 1))
    x = torch.cat(rows)
    q, c = torch.zeros(x.shape, dtype=torch.int8, device="cuda"), torch.zeros(len(x), device="cuda")
    tq.int8_quant_rows(x.cuda(), q, c)
    rq, rc = quantised(x)
    assert torch.equal(c.cpu(), rc) and torch.equal(q.cpu(), rq)


def run_product(counts, d_in, d_out, out, gather=0, wide=0, lead=2, tail=3, seed=3):
    g, od = gen(seed), DT[out]
    off = offsets(counts, lead)
    rows = off[-1] + tail
    x_rows = max(1, rows // 2) if gather else rows
    src = None
    if gather:
        src = torch.randint(0, x_rows * gather, (rows,), generator=g, dtype=I32)
        src[lead] = x_rows * gather          # a row of zeros
        src[rows - tail - 1] = -1
    x, w = codes(g, (x_rows, d_in + wide)), codes(g, (len(counts), d_out, d_in))
    xs = torch.rand(x_rows, generator=g) + 0.01
    ws = torch.rand((len(counts), d_out), generator=g) * 1e-3 + 1e-5
    # rows of y start one element in and are d_out + 1 + wide apart
    flat = torch.full((rows * (d_out + 1 + wide) + 8,), -7.0, dtype=od, device="cuda")
    at = 1 if wide else 0
    y = flat[at:at + rows * (d_out + at + wide)].view(rows, d_out + at + wide)[:, :d_out]
    tq.int8_gemm(x.cuda()[:, :d_in], xs.cuda(), w.cuda(), ws.cuda(), y,
                 off=torch.tensor(off, dtype=I32, device="cuda"), src=None if src is None else src.cuda(),
                 src_div=max(gather, 1))
    got = y.cpu()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        r = torch.arange(lo, hi) if src is None else torch.div(src[lo:hi].long(), max(gather, 1), rounding_mode="floor")
        bad = (r < 0) | (r >= x_rows)
        r = r.clamp(0, x_rows - 1)
        want = product(x[r][:, :d_in], xs[r], w[e], ws[e], od)
        want[bad] = 0
        assert torch.equal(got[lo:hi], want), (e, (got[lo:hi].double() - want.double()).abs().max())
    y[off[0]:off[-1]] = -7.0
    assert (flat == -7).all(), "something beside the rows was written"


@pytest.mark.parametrize("kernel,groups,rows,d_in,d_out", CASES, ids=IDS)
@pytest.mark.parametrize("gather", [0, 3])
def test_every_kernel(kernel, groups, rows, d_in, d_out, gather):
    print(f"[case] int8 {kernel} {groups} {rows} {d_in} {d_out} {gather}", flush=True)
    assert kernel_of(groups, rows, d_in, d_out) == kernel
    if groups == 1:
        run_product([rows - 5], d_in, d_out, "bf16", gather)
    else:
        run_product(ragged(groups, rows, 2, 3), d_in, d_out, "f32" if gather else "f16", gather)


@pytest.mark.parametrize("counts,d_in,d_out", [([1], 4096, 512), ([1], 16, 1), ([2, 0, 1, 3], 144, 13),
                                               ([40, 1, 70], 528, 129), ([3000, 0, 2000], 400, 257),
                                               ([129, 0, 300, 1], 400, 391)])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("wide", [0, 16])
def test_sizes(counts, d_in, d_out, out, wide):
    print(f"[case] int8 product {counts} {d_in} {d_out} {out} {wide}", flush=True)
    run_product(counts, d_in, d_out, out, wide=wide)


@pytest.mark.parametrize("rows", [2, 40, 300])
def test_largest_sums(rows):
    """All codes -128 over the longest row: 128^2 * 131056, just below 2^31."""
    d = 131056
    x, w = torch.full((rows, d), -128, dtype=torch.int8, device="cuda"), torch.full((24, d), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    y = torch.empty((rows, 24), device="cuda")
    tq.int8_gemm(x, torch.ones(rows, device="cuda"), w, torch.ones(24, device="cuda"), y)
    assert (y[:, 1] == -128 * 127 * d).all() and (y[:, [0] + list(range(2, 24))] == 128 * 128 * d).all()


def test_one_matrix_and_special_scales():
    x, w = codes(gen(4), (5, 64)), codes(gen(5), (24, 64))
    xs, ws = torch.tensor([1.0, float("nan"), 2.0 ** -126, 1e30, 0.0]), torch.ones(24)
    ws[3], ws[4] = float("nan"), 2.0 ** 100
    y = torch.empty((5, 24), device="cuda")
    tq.int8_gemm(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), y)
    assert same(y.cpu(), product(x, xs, w, ws, torch.float32))


def test_empty_calls():
    w, ws = torch.ones((1, 40, 256), dtype=torch.int8, device="cuda"), torch.ones((1, 40), device="cuda")
    empty = torch.empty((0, 256), device="cuda")
    q, c = empty.to(torch.int8), torch.empty(0, device="cuda")
    tq.int8_quant_rows(empty, q, c)
    tq.int8_gemm(q, c, w, ws, torch.empty((0, 40), device="cuda"))
    y = torch.full((3, 40), 7.0, device="cuda")
    tq.int8_gemm(q, c, w, ws, y, src=torch.tensor([0, 1, 5], dtype=I32, device="cuda"))
    assert (y == 0).all()


def test_graph_replay_and_streams():
    T, i, o = 33, 1024, 512
    x, w = normal(gen(6), (T, i), 1.0, torch.float16).cuda(), normal(gen(7), (o, i), 0.03, torch.float16).cuda()
    xq, xc = torch.zeros((T, i), dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda")
    wq, wc = torch.zeros((o, i), dtype=torch.int8, device="cuda"), torch.zeros(o, device="cuda")
    y = torch.empty((T, o), device="cuda")

    def step(stream=None):
        tq.int8_quant_rows(w, wq, wc, stream=stream)
        tq.int8_quant_rows(x, xq, xc, stream=stream)
        tq.int8_gemm(xq, xc, wq, wc, y, stream=stream)

    step()
    torch.cuda.synchronize()
    want = y.clone()
    assert torch.equal(want.cpu(), product(xq.cpu(), xc.cpu(), wq.cpu(), wc.cpu(), torch.float32))
    side = torch.cuda.Stream()
    y.fill_(float("nan"))
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        y.fill_(float("nan"))
        xc.zero_()
        torch.randn(1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
