"""Grouped products of sizes that take each of the kernels, at several stages of
k, so that rings of buffers wrap and groups end inside tiles."""
import ctypes

import bit_rank_post_amd as tq

Y, DX, DW, F8 = 0, 1, 2, 3
NAMES = {Y: "y", DX: "dx", DW: "dw", F8: "e4m3"}

# product, kernel (outputs x rows of a workgroup, staged in LDS or not), groups,
# rows, d_in, d_out
CASES = [
    (Y, (16, 16, 0), 7, 40, 520, 136), (Y, (16, 16, 0), 70, 40, 520, 136),
    (Y, (32, 32, 0), 4, 40, 520, 136), (Y, (32, 32, 0), 70, 700, 520, 136),
    (Y, (128, 32, 1), 16, 4200, 520, 136), (Y, (128, 32, 1), 70, 4200, 520, 136),
    (Y, (128, 128, 1), 4, 9000, 520, 136), (Y, (128, 128, 1), 70, 9000, 520, 136),
    (Y, (256, 256, 1), 16, 6000, 520, 1032), (Y, (256, 256, 1), 70, 9000, 520, 2056),
    (DX, (128, 32, 1), 4, 40, 136, 520), (DX, (128, 32, 1), 70, 40, 136, 520),
    (DX, (128, 128, 1), 4, 9000, 136, 520), (DX, (128, 128, 1), 70, 9000, 136, 520),
    (DX, (256, 256, 1), 4, 12000, 1032, 456), (DX, (256, 256, 1), 66, 40000, 2040, 4104),
    (DW, (128, 128, 1), 4, 1900, 136, 264), (DW, (128, 128, 1), 66, 9000, 136, 264),
    (DW, (256, 256, 1), 16, 2100, 520, 1032), (DW, (256, 256, 1), 70, 9000, 264, 520),
    (F8, (16, 16, 0), 7, 40, 912, 136), (F8, (16, 16, 0), 70, 40, 912, 136),
    (F8, (32, 32, 0), 4, 40, 912, 136), (F8, (32, 32, 0), 70, 700, 912, 136),
    (F8, (128, 32, 1), 7, 3100, 912, 136), (F8, (128, 32, 1), 70, 2100, 1040, 136),
    (F8, (128, 128, 1), 4, 9000, 912, 136), (F8, (128, 128, 1), 70, 9000, 912, 136),
    (F8, (256, 256, 1), 40, 6000, 912, 1032), (F8, (256, 256, 1), 1, 4200, 912, 2056),
]
IDS = [f"{NAMES[c[0]]}-{c[1][0]}x{c[1][1]}-{c[2]}g" for c in CASES]


def kernel_of(product, groups, rows, d_in, d_out, act=tq.TQ_F16):
    """(outputs, rows, staged) of the kernel that a product takes (host only)."""
    d = tq.GroupDesc(groups, rows, d_in, d_out, act, 0x10000 if groups > 1 else None, None, 1, rows, 0, 0)
    out = [ctypes.c_int32() for _ in range(3)]
    tq._check("tq_debug_group_kernel", tq.lib().tq_debug_group_kernel(
        ctypes.byref(d), product, *[ctypes.byref(v) for v in out]))
    return tuple(v.value for v in out)


def ragged(groups, rows, lead, tail):
    """Row counts that add up to rows - lead - tail: one group with more than
    twice the average, empty groups and groups of one row among the others."""
    left = rows - lead - tail
    if groups == 1:
        return [left]
    share = [0 if g % 5 == 3 else (1 + g * 37 % 23) for g in range(groups)]
    share[groups // 2] = 3 * sum(share) // groups + 1
    share[-1] = max(share[-1], 1)
    counts = [left * s // sum(share) for s in share]
    if groups > 4:
        counts[1] = min(counts[1], 1)
    counts[groups // 2] += left - sum(counts)
    return counts
