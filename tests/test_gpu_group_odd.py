"""Forward products with any number of outputs and any place of y: odd widths,
rows of y that are not 16-byte aligned, rows of x that are all absent."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.group_cases import kernel_of
from tests.ops_util import DT, check, gen, half_step, normal, offsets

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# outputs below, at and past the widths of fragments, waves and tiles
@pytest.mark.parametrize("d_out", [1, 3, 13, 60, 127, 129, 257, 1001])
@pytest.mark.parametrize("counts,d_in", [([3, 0, 2], 72), ([40, 1, 70], 520), ([3000, 0, 2000], 208)])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("at", [0, 1])
def test_16_bit(d_out, counts, d_in, out, at):
    g, od = gen(41), DT[out]
    off = offsets(counts, 1)
    rows = off[-1] + 2
    print(f"[case] {kernel_of(0, len(counts), rows, d_in, d_out)} {counts} {d_in} {d_out} {out} {at}", flush=True)
    x, w = normal(g, (rows, d_in), 1.0, torch.bfloat16), normal(g, (len(counts), d_out, d_in), 1.0, torch.bfloat16)
    # rows of y start `at` elements in and are d_out + at apart: odd addresses
    flat = torch.full((rows * (d_out + at) + 8,), -7.0, dtype=od, device="cuda")
    y = flat[at:at + rows * (d_out + at)].view(rows, d_out + at)[:, :d_out]
    tq.group_gemm(x.cuda(), w.cuda(), y, off=torch.tensor(off, dtype=torch.int32, device="cuda"))
    got = y.cpu()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        a, b = x[lo:hi].double(), w[e].double().t()
        ref, mag = a @ b, a.abs() @ b.abs()
        check(f"expert {e}", got[lo:hi], ref, d_in * 2.0 ** -23 * mag + half_step(ref, od))
    y[off[0]:off[-1]] = -7.0
    assert (flat == -7).all(), "something beside the rows was written"


@pytest.mark.parametrize("d_out", [1, 13, 127, 129, 257])
@pytest.mark.parametrize("counts,d_in", [([3, 0, 2], 144), ([40, 1, 70], 528), ([3000, 0, 2000], 400)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_8_bit(d_out, counts, d_in, out):
    """Whole numbers up to 15 and scales of powers of two: exact up to the output's rounding."""
    g, od = gen(42), DT[out]
    off = offsets(counts, 1)
    rows, nk, no = off[-1] + 2, -(-d_in // 128), -(-d_out // 128)
    print(f"[case] {kernel_of(3, len(counts), rows, d_in, d_out)} {counts} {d_in} {d_out} {out}", flush=True)
    x = torch.randint(-15, 16, (rows, d_in), generator=g).float()
    w = torch.randint(-15, 16, (len(counts), d_out, d_in), generator=g).float()
    xc = 2.0 ** torch.randint(-3, 1, (rows, nk), generator=g).float()
    wc = 2.0 ** torch.randint(-3, 1, (len(counts), no, nk), generator=g).float()
    flat = torch.full((rows * (d_out + 1) + 8,), -7.0, dtype=od, device="cuda")
    y = flat[1:1 + rows * (d_out + 1)].view(rows, d_out + 1)[:, :d_out]
    tq.fp8_gemm(x.to(E4M3).cuda(), xc.cuda(), w.to(E4M3).cuda(), wc.cuda(), y,
                off=torch.tensor(off, dtype=torch.int32, device="cuda"))
    got = y.cpu()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        a = x[lo:hi].double() * xc[lo:hi].double().repeat_interleave(128, 1)[:, :d_in]
        s = wc[e].double().repeat_interleave(128, 0)[:d_out].repeat_interleave(128, 1)[:, :d_in]
        # whole multiples of 2^-6 below 528 * 225 < 2^17: exact in f32
        assert torch.equal(got[lo:hi], (a @ (w[e].double() * s).t()).to(od)), e
    y[off[0]:off[-1]] = -7.0
    assert (flat == -7).all(), "something beside the rows was written"


def test_no_rows_of_x_at_all():
    """Every index lies outside an x without rows: rows of zeros."""
    src = torch.tensor([0, 1, 5], dtype=torch.int32, device="cuda")
    w, y = torch.ones((1, 24, 64), dtype=torch.float16, device="cuda"), torch.full((3, 24), 7.0, device="cuda")
    x = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    tq.group_gemm(x, w, y, src=src)
    assert (y == 0).all()
    dw = torch.full((1, 24, 64), 7.0, device="cuda")
    tq.group_gemm_dw(torch.ones((3, 24), dtype=torch.float16, device="cuda"), x, dw, src=src)
    assert (dw == 0).all()
    y.fill_(7.0)
    tq.fp8_gemm(x.to(E4M3), torch.empty((0, 1), device="cuda"), w.to(E4M3), torch.ones((1, 1, 1), device="cuda"), y,
                src=src)
    assert (y == 0).all()
