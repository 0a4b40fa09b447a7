"""Sizes of the layer for a few tokens that take each of its kernels, with many
slots of one expert among few of the others."""
import ctypes
import math

import torch

import bit_rank_post_amd as tq
from tests.int8_cases import codes
from tests.ops_util import gen, normal

# columns, up (outputs, waves), down, then experts, tokens, topk, d, ff; slots of one expert
CASES16 = [
    (16, (16, 4), (32, 8), 8, 9, 2, 136, 72, 17),
    (16, (16, 4), (16, 4), 64, 20, 4, 264, 40, 33),
    (16, (32, 4), (32, 8), 4, 16, 3, 2048, 4104, 33),
    (16, (32, 4), (16, 4), 60, 16, 4, 2056, 296, 33),
    (16, (32, 8), (32, 8), 4, 9, 2, 2048, 264, 17),
    (16, (32, 8), (16, 4), 8, 32, 2, 2048, 264, 50),
    (16, (16, 8), (32, 8), 2, 9, 2, 4072, 200, 17),
    (16, (16, 8), (16, 4), 4, 16, 4, 4104, 200, 49),
    (16, (16, 4), (16, 4), 128, 16, 8, 144, 24, 64),
    (32, (32, 4), (64, 8), 2, 30, 2, 136, 72, 33),
    (32, (32, 4), (64, 8), 1, 24, 4, 264, 104, 96),
    (32, (32, 4), (64, 8), 3, 17, 4, 1032, 136, 65),
    (64, (32, 4), (64, 4), 2, 40, 2, 136, 72, 65),
    (64, (32, 4), (64, 4), 1, 40, 4, 264, 104, 160),
    (1, (16, 4), (16, 16), 8, 1, 4, 264, 72, 3), (1, (16, 8), (16, 16), 6, 1, 2, 2048, 264, 2),
    (1, (16, 8), (16, 8), 5, 1, 3, 4104, 200, 1),
]
CASES8 = [
    (16, (16, 4), (32, 8), 8, 9, 2, 144, 80, 17),
    (16, (16, 4), (32, 4), 64, 20, 4, 272, 48, 33),
    (16, (32, 4), (32, 8), 4, 16, 3, 4000, 4112, 33),
    (16, (32, 4), (32, 4), 64, 16, 4, 4000, 272, 33),
    (16, (32, 8), (32, 8), 4, 9, 2, 4000, 272, 17),
    (16, (32, 8), (32, 4), 8, 32, 2, 4000, 272, 50),
    (16, (16, 8), (32, 8), 2, 9, 2, 8080, 208, 17),
    (16, (16, 8), (32, 4), 4, 16, 4, 8208, 208, 49),
    (16, (16, 4), (32, 4), 128, 16, 8, 144, 32, 64),
    (32, (32, 4), (64, 8), 2, 30, 2, 144, 80, 33),
    (32, (32, 4), (64, 8), 1, 24, 4, 272, 112, 96),
    (32, (32, 4), (64, 8), 3, 17, 4, 1040, 144, 65),
    (64, (32, 4), (64, 4), 2, 40, 2, 144, 80, 65),
    (64, (32, 4), (64, 4), 1, 40, 4, 272, 112, 160),
    (1, (16, 4), (16, 16), 8, 1, 4, 272, 80, 3), (1, (16, 8), (16, 16), 6, 1, 2, 4000, 272, 2),
    (1, (16, 8), (16, 8), 5, 1, 3, 4112, 208, 1),
]


def kernels_of(T, topk, experts, d, ff, int8):
    """Columns, up and down kernel (outputs, waves) that a call takes (host only)."""
    c, up, down = ctypes.c_int32(), (ctypes.c_int32 * 2)(), (ctypes.c_int32 * 2)()
    tq._check("tq_debug_experts_kernels",
              tq.lib().tq_debug_experts_kernels(T, topk, experts, d, ff, int8, ctypes.byref(c), up, down))
    return c.value, tuple(up), tuple(down)


def skewed(E, T, k, d, ff, hot, dtype, int8, seed, whole=False):
    """x, ids, w, w_up, w_down, s_up, s_down: `hot` slots of one expert, at random
    places, the others' at random, one of them outside the experts.  whole: x and
    w_up whole numbers (w_up of 16 bits times a power of two), so that the sums of
    their products are exact in f32 in any order."""
    g = gen(seed)
    e = int(torch.randint(0, E, (1,), generator=g))
    ids = torch.randint(0, max(E - 1, 1), (T * k,), generator=g)
    if E > 1:
        ids[ids >= e] += 1
    at = torch.randperm(T * k, generator=g)
    ids[at[:hot]] = e
    if hot < T * k:
        ids[at[-1]] = -1
    x, w = normal(g, (T, d), 1.0, dtype), torch.softmax(torch.randn((T, k), generator=g), 1)
    s_up = s_down = None
    if int8:
        w_up, w_down = codes(g, (E, 2 * ff, d)), codes(g, (E, d, ff))
        s_up = (torch.rand((E, 2 * ff), generator=g) + 0.5) * d ** -0.5 / 74
        s_down = (torch.rand((E, d), generator=g) + 0.5) * ff ** -0.5 / 74
    else:
        w_up, w_down = normal(g, (E, 2 * ff, d), d ** -0.5, dtype), normal(g, (E, d, ff), ff ** -0.5, dtype)
    if whole:
        # (codes -2 .. 2 and -128 .. 127: below 2^21 and 2^22 of at most 8208 terms)
        x = torch.randint(-2, 3, (T, d), generator=g).to(dtype)
        if not int8:
            w_up = torch.randint(-2, 3, w_up.shape, generator=g, dtype=torch.int8).to(dtype) * 2.0 ** -round(math.log2(2 * d ** 0.5))
    return x, ids.view(T, k).to(torch.int32), w, w_up, w_down, s_up, s_down
