"""8-bit quantisation and products with a scale for each block of 128, against
the definition in 64 bits."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import DT, check, gen, half_step, normal, offsets

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def ref_scale(amax):
    """fl32 of amax / 448 (64-bit division rounds to the same f32), at least
    the smallest normal, 1 for zero, not a number for that."""
    c = (amax.double() / 448).float().clamp(min=2.0 ** -126)
    return torch.where(amax == 0, torch.ones_like(c), c)


def same(a, b):
    """Equal values, not-a-number in the same places."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(3.5), b.nan_to_num(3.5))


def ref_codes(v, c):
    """Values of e4m3 codes of fl32(v / c), ties to even."""
    f = (v.double() / c.double()).float().double()
    exp = torch.frexp(f).exponent.double() - 1
    step = torch.exp2(exp.clamp(min=-6) - 3)
    return torch.round(f / step) * step


def quant_rows_ref(x):
    rows, d = x.shape
    nb = -(-d // 128)
    pad = torch.zeros((rows, nb * 128))
    pad[:, :d] = x.float()
    blk = pad.view(rows, nb, 128)
    c = ref_scale(blk.abs().amax(2))
    return ref_codes(blk, c[:, :, None]).view(rows, -1)[:, :d], c


def quant_blocks_ref(w):
    G, o, i = w.shape
    no, ni = -(-o // 128), -(-i // 128)
    pad = torch.zeros((G, no * 128, ni * 128))
    pad[:, :o, :i] = w.float()
    blk = pad.view(G, no, 128, ni, 128)
    c = ref_scale(blk.abs().amax((2, 4)))
    return ref_codes(blk, c[:, :, None, :, None]).view(G, no * 128, -1)[:, :o, :i], c


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,d,wide", [(1, 16, 0), (1, 128, 0), (3, 144, 8), (17, 4096, 0), (300, 272, 16)])
def test_quant_rows(dtype, rows, d, wide):
    print(f"[case] quant rows {dtype} {rows} {d} {wide}", flush=True)
    x = normal(gen(1), (rows, d + wide), 3.0, DT[dtype])
    x[0, :16] = 0
    if rows > 2:
        x[2] = 0
        x[1, :128] *= 2.0 ** -12
    q = torch.zeros((rows, d), dtype=E4M3, device="cuda")
    c = torch.zeros((rows, -(-d // 128)), device="cuda")
    xd = x.cuda()
    tq.fp8_quant_rows(xd[:, :d], q, c)
    rq, rc = quant_rows_ref(x[:, :d])
    assert torch.equal(c.cpu(), rc)
    assert torch.equal(q.float().double().cpu(), rq)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("G,o,i", [(1, 1, 16), (2, 130, 144), (3, 128, 256), (1, 520, 1408)])
def test_quant_blocks(dtype, G, o, i):
    print(f"[case] quant blocks {dtype} {G} {o} {i}", flush=True)
    w = normal(gen(2), (G, o, i), 0.02, DT[dtype])
    q = torch.zeros((G, o, i), dtype=E4M3, device="cuda")
    c = torch.zeros((G, -(-o // 128), -(-i // 128)), device="cuda")
    tq.fp8_quant_blocks(w.cuda(), q, c)
    rq, rc = quant_blocks_ref(w)
    assert torch.equal(c.cpu(), rc)
    assert torch.equal(q.float().double().cpu(), rq)


def test_quant_special_values():
    x = torch.zeros((6, 256))
    x[0, :128] = 1e-45                    # below the smallest normal scale
    x[1, :128] = torch.linspace(-3e38, 3e38, 128)
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    x[4, :128] = 2.0 ** -149 * 448 * 1000
    x[5, 0], x[5, 1] = -0.0, -448.0
    q, c = torch.zeros((6, 256), dtype=E4M3, device="cuda"), torch.zeros((6, 2), device="cuda")
    tq.fp8_quant_rows(x.cuda(), q, c)
    deq = q.float().cpu() * c.cpu().repeat_interleave(128, 1)
    assert torch.isnan(deq[2, 5]) and torch.isnan(deq[3, 128:]).all()
    assert torch.isfinite(deq[3, :128]).all() and torch.isfinite(deq[2, 128:]).all()
    rest = [0, 1, 4, 5]
    rq, rc = quant_rows_ref(x[rest])
    # (linspace's own step overflows, so row 1 holds not-a-number)
    assert same(c.cpu()[rest], rc) and same(q.float().double().cpu()[rest], rq)
    big = torch.linspace(-3e0, 3e0, 128)[None] * 1e38
    q, c = torch.zeros((1, 128), dtype=E4M3, device="cuda"), torch.zeros((1, 1), device="cuda")
    tq.fp8_quant_rows(big.cuda(), q, c)
    rq, rc = quant_rows_ref(big)
    assert torch.equal(c.cpu(), rc) and torch.equal(q.float().double().cpu(), rq)
    xh = torch.full((1, 16), 65504.0, dtype=torch.float16, device="cuda")
    q, c = torch.zeros((1, 16), dtype=E4M3, device="cuda"), torch.zeros((1, 1), device="cuda")
    tq.fp8_quant_rows(xh, q, c)
    assert (q.float() == 448).all()


def product_bound(x, xc, w, wc, lo, hi, e, src, div, out, whole):
    """Reference and bound.  The matrix unit adds 8 products at a time: it cuts
    each at 2^-13 of the power of two below the largest of the 8 (so what it
    drops is less than 2^-13 of that largest product, 7 times, and nothing of
    the largest) and adds the results in f32.  With integers up to 15 nothing
    is below the cut (the largest is less than 2^8, so it is below 2^-5), and a
    block's sum is exact (128 * 225 < 2^24).  Then the block's product with
    fl32(xs ws) (two roundings) and the sum over nb blocks: (nb + 2) 2^-23 of
    the magnitudes, and 128 more inside a block where it is not exact."""
    d = x.shape[1]
    rows = torch.arange(lo, hi) if src is None else src[lo:hi].long() // div
    a = x.double()[rows] * xc.double()[rows].repeat_interleave(128, 1)[:, :d]
    s = wc[e].double().repeat_interleave(128, 0)[:w.shape[1]].repeat_interleave(128, 1)[:, :d]
    b = w[e].double() * s
    ref, mag = a @ b.t(), a.abs() @ b.abs().t()
    nb = -(-d // 128)
    unit = 0.0 if whole else 7 * 2.0 ** -13 + 128 * 2.0 ** -23
    return ref, (unit + (nb + 2) * 2.0 ** -23) * mag + half_step(ref, out)


@pytest.mark.parametrize("counts,d_in,d_out", [
    ([1], 4096, 512), ([1], 16, 8), ([2, 0, 1, 3], 144, 136), ([16, 17, 0, 15, 33], 272, 200),
    ([64, 100], 2048, 264), ([129, 0, 300, 1], 400, 392), ([1500], 512, 1100), ([700, 5, 900], 1408, 2048),
    ([4100], 160, 4104)])
@pytest.mark.parametrize("kind", ["plain", "gather", "strided"])
@pytest.mark.parametrize("values", ["normal", "whole"])
def test_product(counts, d_in, d_out, kind, values):
    print(f"[case] fp8 product {counts} {d_in} {d_out} {kind} {values}", flush=True)
    out = {"plain": torch.bfloat16, "gather": torch.float32, "strided": torch.float16}[kind]
    gather, wide = (2 if kind == "gather" else 0), (16 if kind == "strided" else 0)
    g = gen(3)
    off = offsets(counts, 2)
    rows = off[-1] + 3
    x_rows = max(1, rows // 2) if gather else rows
    src = torch.randint(0, x_rows * 2, (rows,), generator=g, dtype=torch.int32) if gather else None
    x = torch.full((x_rows, d_in + wide), float("nan")).to(E4M3)
    x[:, :d_in] = normal(g, (x_rows, d_in), 60.0, torch.float32).clamp(-448, 448).to(E4M3)
    xc = torch.rand((x_rows, -(-d_in // 128)), generator=g) + 0.01
    w = normal(g, (len(counts), d_out, d_in), 60.0, torch.float32).clamp(-448, 448).to(E4M3)
    wc = torch.rand((len(counts), -(-d_out // 128), -(-d_in // 128)), generator=g) * 1e-3 + 1e-5
    if values == "whole":
        x[:, :d_in] = torch.randint(-15, 16, (x_rows, d_in), generator=g).float().to(E4M3)
        w = torch.randint(-15, 16, w.shape, generator=g).float().to(E4M3)
    y = torch.full((rows, d_out + wide), -7.0, dtype=out, device="cuda")
    xd = x.cuda()
    tq.fp8_gemm(xd[:, :d_in], xc.cuda(), w.cuda(), wc.cuda(), y[:, :d_out],
                off=torch.tensor(off, dtype=torch.int32, device="cuda"),
                src=None if src is None else src.cuda(), src_div=max(gather, 1))
    torch.cuda.synchronize()
    got, xf, wf = y.cpu(), x[:, :d_in].float(), w.float()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        ref, tol = product_bound(xf, xc, wf, wc, lo, hi, e, src, max(gather, 1), out, values == "whole")
        check(f"expert {e}", got[lo:hi, :d_out], ref, tol)
    assert (got[:off[0]] == -7).all() and (got[off[-1]:] == -7).all() and (got[:, d_out:] == -7).all()


def test_quantised_product_of_one_matrix():
    """Quantise and multiply, one matrix, no groups: each value is off by half
    an e4m3 step at most, 2^-4 of it, or half the smallest step of its block."""
    T, i, o = 70, 528, 300
    x, w = normal(gen(4), (T, i), 1.0, torch.bfloat16), normal(gen(5), (o, i), 0.05, torch.bfloat16)
    xq, xc = torch.zeros((T, i), dtype=E4M3, device="cuda"), torch.zeros((T, 5), device="cuda")
    wq, wc = torch.zeros((o, i), dtype=E4M3, device="cuda"), torch.zeros((3, 5), device="cuda")
    tq.fp8_quant_rows(x.cuda(), xq, xc)
    tq.fp8_quant_blocks(w.cuda(), wq, wc)
    y = torch.empty((T, o), device="cuda")
    tq.fp8_gemm(xq, xc, wq, wc, y)
    a, b = x.double().abs(), w.double().abs()
    sx = xc.cpu().double().repeat_interleave(128, 1)[:, :i]
    sw = wc.cpu().double().repeat_interleave(128, 0)[:o].repeat_interleave(128, 1)[:, :i]
    # |q c - v| <= v / 16 + c 2^-10 (half the subnormal step 2^-9); the matrix
    # unit's cut (7 2^-13 of a @ b, 0.7 % of what two v / 16 give), the f32
    # divisions and sums add less than 1 % to that
    ea, eb = a / 16 + sx * 2.0 ** -10, b / 16 + sw * 2.0 ** -10
    tol = 1.01 * (ea @ b.t() + a @ eb.t() + ea @ eb.t())
    check("y", y, x.double() @ w.double().t(), tol)


def test_special_values_and_empty_calls():
    x, w = torch.ones((3, 256)).to(E4M3), torch.ones((1, 40, 256), device="cuda").to(E4M3)
    x[1, 200] = float("nan")
    xc, wc = torch.ones((3, 2), device="cuda"), torch.ones((1, 1, 2), device="cuda")
    y = torch.empty((3, 40), device="cuda")
    tq.fp8_gemm(x.cuda(), xc, w, wc, y)
    assert (y[0] == 256).all() and torch.isnan(y[1]).all() and (y[2] == 256).all()
    src = torch.tensor([2, -1, 3], dtype=torch.int32, device="cuda")     # a row of zeros outside x
    tq.fp8_gemm(x.cuda(), xc, w, wc, y, src=src)
    assert (y[0] == 256).all() and (y[1:] == 0).all()
    empty = torch.empty((0, 256), device="cuda")
    tq.fp8_quant_rows(empty, empty.to(E4M3), torch.empty((0, 2), device="cuda"))
    tq.fp8_gemm(empty.to(E4M3), torch.empty((0, 2), device="cuda"), w, wc, torch.empty((0, 40), device="cuda"))


def test_graph_replay():
    T, i, o = 33, 1024, 512
    x, w = normal(gen(6), (T, i), 1.0, torch.float16).cuda(), normal(gen(7), (o, i), 0.03, torch.float16).cuda()
    xq, xc = torch.zeros((T, i), dtype=E4M3, device="cuda"), torch.zeros((T, 8), device="cuda")
    wq, wc = torch.zeros((o, i), dtype=E4M3, device="cuda"), torch.zeros((4, 8), device="cuda")
    y = torch.empty((T, o), device="cuda")

    def step():
        tq.fp8_quant_blocks(w, wq, wc)
        tq.fp8_quant_rows(x, xq, xc)
        tq.fp8_gemm(xq, xc, wq, wc, y)

    step()
    torch.cuda.synchronize()
    want = y.clone()
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


def test_quotients_are_correctly_rounded():
    """Codes of many quotients next to the borders between codes, at scales from
    the smallest to the largest: equal to the definition, one by one."""
    g = gen(8)
    rows = []
    for e in (-126, -120, -101, -100, -99, -60, -10, 0, 7, 60, 100, 118):
        amax = (1 + torch.rand((64, 1), generator=g)) * 2.0 ** e * 448
        c = ref_scale(amax.clamp(max=3e38))
        # the middle of two codes, and its neighbours in f32
        code = torch.randint(1, 127, (64, 128), generator=g).float()
        man, exp = code % 8, torch.floor(code / 8)
        val = torch.where(exp > 0, (1 + (man + 0.5) / 8) * torch.exp2(exp - 7), (man + 0.5) * 2.0 ** -9)
        x = (val.clamp(max=447) * c).to(torch.float32)
        step = torch.randint(-2, 3, (64, 128), generator=g, dtype=torch.int32)
        x = (x.view(torch.int32) + step).clamp(min=0).view(torch.float32)
        x[:, 0] = amax[:, 0].clamp(max=3e38)
        rows.append(x)
    x = torch.cat(rows)
    q, c = torch.zeros(x.shape, dtype=E4M3, device="cuda"), torch.zeros((len(x), 1), device="cuda")
    tq.fp8_quant_rows(x.cuda(), q, c)
    rq, rc = quant_rows_ref(x)
    assert torch.equal(c.cpu(), rc)
    assert torch.equal(q.float().double().cpu(), rq)
