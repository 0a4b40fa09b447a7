"""Products of 8-bit integers of sizes that take each of the kernels, and their
exact results: the sum of codes is a whole number below 2^31, and what follows
it is one f32 operation after the other."""
import ctypes

import torch

import bit_rank_post_amd as tq

# kernel (outputs x rows of a workgroup, staged in LDS or not), groups, rows, d_in, d_out
CASES = [
    ((16, 16, 0), 7, 40, 912, 136), ((16, 16, 0), 70, 40, 912, 136),
    ((32, 32, 0), 4, 40, 912, 136), ((32, 32, 0), 70, 700, 912, 136),
    ((128, 32, 1), 30, 4200, 1040, 136), ((128, 32, 1), 70, 4200, 1040, 136),
    ((128, 128, 1), 4, 9000, 912, 520), ((128, 128, 1), 70, 9000, 912, 520),
    ((256, 256, 1), 16, 9000, 1040, 1032), ((256, 256, 1), 66, 20000, 912, 1032), ((256, 256, 1), 1, 4200, 912, 4104),
]
IDS = [f"{c[0][0]}x{c[0][1]}-{c[1]}g" for c in CASES]


def kernel_of(groups, rows, d_in, d_out):
    """(outputs, rows, staged) of the kernel that a product takes (host only)."""
    d = tq.GroupDesc(groups, rows, d_in, d_out, tq.TQ_F16, 0x10000 if groups > 1 else None, None, 1, rows, 0, 0)
    out = [ctypes.c_int32() for _ in range(3)]
    tq._check("tq_debug_int8_kernel", tq.lib().tq_debug_int8_kernel(ctypes.byref(d), *[ctypes.byref(v) for v in out]))
    return tuple(v.value for v in out)


def codes(g, shape, lo=-128):
    return torch.randint(lo, 128, shape, generator=g, dtype=torch.int32).to(torch.int8)


def product(x, xs, w, ws, dtype):
    """fl(fl(fl(sum) ws) xs), rounded to dtype.  Sums of whole numbers below 2^53
    are exact in f64 in any order."""
    acc = x.double() @ w.double().t()
    return (acc.float() * ws[None, :] * xs[:, None]).to(dtype)


def ref_scale(amax):
    """fl32 of amax / 127, at least the smallest normal, 1 for zero, NaN for no number."""
    c = (amax.double() / 127).float().clamp(min=2.0 ** -126)
    c = torch.where(torch.isfinite(amax), c, torch.full_like(c, float("nan")))
    return torch.where(amax == 0, torch.ones_like(c), c)


def quantised(x):
    """Codes and scales of the rows of x, by the definition."""
    x = x.float()
    c = ref_scale(x.abs().amax(1))
    q = torch.round((x.double() / c.double()[:, None]).float())
    return torch.where(torch.isnan(c)[:, None], torch.zeros_like(q), q).to(torch.int8), c
