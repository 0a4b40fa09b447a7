"""Refusals of the int8 products, SwiGLU, the sum over slots and the layer for a
few tokens, on the CPU: every check runs on the host before any launch (the
pointers passed here are never dereferenced)."""
import ctypes
import os

import pytest

import bit_rank_post_amd as tq

P, Q, R = 0x10000, 0x20000, 0x30000       # aligned addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(tq.LIB_PATH):
        pytest.skip("libtileq.so not built")
    return tq.lib()


def fill(cls, base, kw):
    base = dict(base, **kw)
    vals = []
    for name, typ in cls._fields_:
        v = base[name]
        vals.append((tq.Rows(*v) if isinstance(v, tuple) else tq.Rows(v, 0)) if typ is tq.Rows else v)
    return cls(*vals)


def refused(L, status, code, text):
    assert status == code, (status, L.tq_last_error())
    assert text in L.tq_last_error(), L.tq_last_error()


def group(**kw):
    return fill(tq.GroupDesc, dict(groups=2, rows=64, d_in=128, d_out=64, act=99, off=P, src=None, src_div=1,
                                   x_rows=64, ldx=0, ldy=0), kw)


@pytest.mark.parametrize("kw,code,text", [
    (dict(groups=0), 2, b"groups = 0"), (dict(groups=1025), 2, b"groups"), (dict(rows=-1), 2, b"rows = -1"),
    (dict(off=None), 1, b"off is NULL"), (dict(d_in=0), 2, b"d_in"), (dict(d_in=136), 2, b"d_in"),
    (dict(d_in=131072), 5, b"131072"), (dict(d_out=0), 2, b"d_out"), (dict(ldx=112), 2, b"ldx"), (dict(ldx=136), 2, b"ldx"),
    (dict(ldy=56), 2, b"ldy"), (dict(ldx=(1 << 21) + 16), 5, b"stride"), (dict(src=P, src_div=0), 2, b"src_div"),
    (dict(src=P, x_rows=-1), 2, b"x_rows"), (dict(src=P, x_rows=1 << 24), 5, b"gathered"),
    (dict(rows=2 ** 31 - 1), 5, b"rows"),
])
def test_int8_gemm_descriptor(L, kw, code, text):
    d = ctypes.byref(group(**kw))
    refused(L, L.tq_int8_gemm(d, P, P, Q, P, R, 0, None), code, text)
    v = [ctypes.byref(ctypes.c_int32()) for _ in range(3)]
    refused(L, L.tq_debug_int8_kernel(d, *v), code, text)


def test_int8_gemm_pointers(L):
    d, args = ctypes.byref(group()), [P, P + 64, Q, Q + 64, R]
    refused(L, L.tq_int8_gemm(None, *args, 0, None), 1, b"descriptor")
    refused(L, L.tq_int8_gemm(d, *args, 3, None), 1, b"output dtype")
    for i in range(5):
        a = list(args)
        a[i] = None
        refused(L, L.tq_int8_gemm(d, *a, 0, None), 1, b"NULL")
    for i, off in ((0, 8), (1, 2), (2, 4), (3, 1)):
        a = list(args)
        a[i] += off
        refused(L, L.tq_int8_gemm(d, *a, 0, None), 1, b"aligned")
    for i in range(4):
        a = list(args)
        a[4] = a[i]
        refused(L, L.tq_int8_gemm(d, *a, 0, None), 1, b"operands")
    assert L.tq_int8_gemm(ctypes.byref(group(rows=0)), None, None, None, None, None, 0, None) == 0
    assert L.tq_debug_int8_kernel(None, *[ctypes.byref(ctypes.c_int32()) for _ in range(3)]) == 1
    for i in range(3):
        v = [ctypes.byref(ctypes.c_int32()) for _ in range(3)]
        v[i] = None
        assert L.tq_debug_int8_kernel(d, *v) == 1


def test_int8_quant_rows(L):
    f = L.tq_int8_quant_rows
    for args, code, text in (
            ((P, 3, 4, 128, 0, Q, R), 1, b"x_dtype"), ((P, 0, -1, 128, 0, Q, R), 2, b"rows"),
            ((P, 0, 4, 120, 0, Q, R), 2, b"d = 120"), ((P, 0, 4, 0, 0, Q, R), 2, b"d = 0"),
            ((P, 0, 4, 131072, 0, Q, R), 5, b"131072"), ((P, 0, 4, 128, 100, Q, R), 2, b"stride"),
            ((P, 0, 4, 128, 132, Q, R), 2, b"stride"), ((P, 2, 4, 128, 130, Q, R), 2, b"stride"),
            ((None, 0, 4, 128, 0, Q, R), 1, b"NULL"), ((P, 0, 4, 128, 0, None, R), 1, b"NULL"),
            ((P, 0, 4, 128, 0, Q, None), 1, b"NULL"), ((P + 2, 0, 4, 128, 0, Q, R), 1, b"aligned"),
            ((P, 0, 4, 128, 0, Q + 8, R), 1, b"aligned"), ((P, 0, 4, 128, 0, Q, R + 2), 1, b"aligned"),
            ((P, 0, 4, 128, 0, P, R), 1, b"operands"), ((P, 0, 4, 128, 0, Q, P), 1, b"operands"),
            ((P, 0, 4, 128, 0, Q, Q), 1, b"operands")):
        refused(L, f(*args, None), code, text)
    assert f(None, 0, 0, 128, 0, None, None, None) == 0


def swiglu(**kw):
    return fill(tq.SwigluDesc, dict(rows=4, ff=64, groups=0, a_dtype=0, h_dtype=0, off=None, a=P, h=Q, dh=R,
                                    da=P + 0x8000), kw)


@pytest.mark.parametrize("kw,code,text", [
    (dict(rows=-1), 2, b"rows = -1"), (dict(ff=0), 2, b"ff = 0"), (dict(ff=12), 2, b"ff = 12"),
    (dict(ff=(1 << 24) + 8), 2, b"ff"), (dict(a_dtype=3), 1, b"dtype"), (dict(h_dtype=-1), 1, b"dtype"),
    (dict(off=P), 2, b"groups = 0"), (dict(off=P + 2, groups=3), 1, b"off"), (dict(a=None), 1, b"a is NULL"),
    (dict(a=P + 8), 1, b"a not 16"), (dict(a=(P, 120)), 2, b"of a"), (dict(a=(P, 132)), 2, b"of a"),
])
def test_swiglu_all(L, kw, code, text):
    d = ctypes.byref(swiglu(**kw))
    refused(L, L.tq_swiglu(d, None), code, text)
    refused(L, L.tq_swiglu_int8(d, Q, R, None), code, text)
    refused(L, L.tq_swiglu_grad(d, None), code, text)


def test_swiglu_each(L):
    for f in (lambda: L.tq_swiglu(None, None), lambda: L.tq_swiglu_int8(None, Q, R, None),
              lambda: L.tq_swiglu_grad(None, None)):
        assert f() == 1
    for kw, code, text in ((dict(h=None), 1, b"h is NULL"), (dict(h=Q + 2), 1, b"h not"), (dict(h=(Q, 60)), 2, b"of h"),
                           (dict(h=P), 1, b"h in place of a"), (dict(h=(P, 128), h_dtype=1), 1, b"h in place of a")):
        refused(L, L.tq_swiglu(ctypes.byref(swiglu(**kw)), None), code, text)
    for kw, code, text in ((dict(dh=None), 1, b"dh is NULL"), (dict(da=None), 1, b"da is NULL"),
                           (dict(da=(P, 136)), 1, b"da in place of a"), (dict(da=(Q, 100)), 2, b"of da"),
                           (dict(h=(R, 72)), 1, b"h in place of dh"), (dict(h=R, h_dtype=2), 1, b"h in place of dh"),
                           (dict(h=P), 1, b"operands"), (dict(da=R), 1, b"operands"), (dict(h=P + 0x8000), 1, b"operands"),
                           (dict(dh=R + 4), 1, b"dh not")):
        refused(L, L.tq_swiglu_grad(ctypes.byref(swiglu(**kw)), None), code, text)
    d = ctypes.byref(swiglu())
    for q, c, code, text in ((None, R, 1, b"NULL"), (Q, None, 1, b"NULL"), (Q + 8, R, 1, b"aligned"),
                             (Q, R + 1, 1, b"aligned"), (P, R, 1, b"operands"), (Q, P, 1, b"operands"), (Q, Q, 1, b"operands")):
        refused(L, L.tq_swiglu_int8(d, q, c, None), code, text)
    refused(L, L.tq_swiglu_int8(ctypes.byref(swiglu(ff=72)), Q, R, None), 2, b"multiple of 16")
    refused(L, L.tq_swiglu_int8(ctypes.byref(swiglu(ff=131072)), Q, R, None), 5, b"131072")
    none = ctypes.byref(swiglu(rows=0, a=None, h=None, dh=None, da=None))
    assert L.tq_swiglu(none, None) == 0 and L.tq_swiglu_grad(none, None) == 0
    assert L.tq_swiglu_int8(none, None, None, None) == 0


def combine(**kw):
    return fill(tq.CombineDesc, dict(T=4, topk=2, d=64, rows=8, z_dtype=0, y_dtype=0, inv=P, w=P + 64, z=Q, y=R, add=None,
                                     dy=R + 0x8000, dz=Q + 0x8000, dw=P + 128), kw)


@pytest.mark.parametrize("kw,code,text", [
    (dict(T=-1), 2, b"T = -1"), (dict(rows=-1), 2, b"rows = -1"), (dict(topk=0), 2, b"topk = 0"),
    (dict(T=1 << 29, topk=2), 5, b"2^30"), (dict(d=0), 2, b"d = 0"), (dict(d=20), 2, b"d = 20"),
    (dict(d=(1 << 24) + 8), 2, b"d = "), (dict(z_dtype=4), 1, b"dtype"), (dict(y_dtype=3), 1, b"dtype"),
    (dict(inv=None), 1, b"inv is NULL"), (dict(inv=P + 2), 1, b"aligned"), (dict(w=P + 1), 1, b"aligned"),
    (dict(z=None), 1, b"z is NULL"), (dict(z=Q + 8), 1, b"z not"), (dict(z=(Q, 56)), 2, b"of z"),
])
def test_combine_both(L, kw, code, text):
    d = ctypes.byref(combine(**kw))
    refused(L, L.tq_combine(d, None), code, text)
    refused(L, L.tq_combine_grad(d, None), code, text)


def test_combine_each(L):
    assert L.tq_combine(None, None) == 1 and L.tq_combine_grad(None, None) == 1
    for kw, code, text in ((dict(y=None), 1, b"y is NULL"), (dict(y=(R, 68)), 2, b"of y"), (dict(add=R + 0x4002), 1, b"add not"),
                           (dict(add=(R, 72)), 1, b"y in place of add"), (dict(y=Q), 1, b"operands"),
                           (dict(y=P + 64), 1, b"operands")):
        refused(L, L.tq_combine(ctypes.byref(combine(**kw)), None), code, text)
    for kw, code, text in ((dict(dy=None), 1, b"dy is NULL"), (dict(dz=None, dw=None), 1, b"neither"),
                           (dict(dz=(Q, 72)), 1, b"dz in place of z"), (dict(dz=(Q + 0x8000, 66)), 2, b"of dz"),
                           (dict(dz=R + 0x8000), 1, b"operands"), (dict(dw=P + 64), 1, b"operands"),
                           (dict(dw=P + 130), 1, b"aligned")):
        refused(L, L.tq_combine_grad(ctypes.byref(combine(**kw)), None), code, text)
    none = ctypes.byref(combine(T=0, inv=None, w=None, z=None, y=None, dy=None, dz=None, dw=None))
    assert L.tq_combine(none, None) == 0 and L.tq_combine_grad(none, None) == 0


def experts(**kw):
    return fill(tq.ExpertsDesc, dict(T=4, topk=2, experts=8, d=64, ff=32, act=0, y_dtype=0, ids=P, w=P + 64, w_up=Q,
                                     w_down=Q + 0x8000, s_up=None, s_down=None, x=R, y=R + 0x8000, add=None), kw)


@pytest.mark.parametrize("kw,code,text", [
    (dict(T=-1), 2, b"T = -1"), (dict(topk=0), 2, b"topk"), (dict(topk=33), 2, b"topk"), (dict(experts=0), 2, b"experts"),
    (dict(experts=1025), 2, b"experts"), (dict(d=0), 2, b"d = 0"), (dict(d=68), 2, b"d = 68"), (dict(d=65544), 2, b"d = "),
    (dict(ff=36), 2, b"ff = 36"), (dict(ff=65544), 2, b"ff"), (dict(T=513), 5, b"1024 slots"), (dict(act=2), 1, b"act"),
    (dict(y_dtype=3), 1, b"y_dtype"), (dict(s_up=P), 1, b"go together"), (dict(s_down=P), 1, b"go together"),
    (dict(s_up=P, s_down=P, d=72), 2, b"multiple of 16"), (dict(s_up=P, s_down=P, ff=40), 2, b"multiple of 16"),
    (dict(s_up=P + 2, s_down=P), 1, b"aligned"), (dict(x=None), 1, b"x is NULL"), (dict(x=R + 8), 1, b"x not"),
    (dict(x=(R, 60)), 2, b"of x"), (dict(x=(R, 1 << 28)), 5, b"2^31"), (dict(y=None), 1, b"NULL"),
    (dict(ids=None), 1, b"NULL"), (dict(w=None), 1, b"NULL"), (dict(w_up=None), 1, b"NULL"), (dict(w_down=None), 1, b"NULL"),
    (dict(w_up=Q + 8), 1, b"aligned"), (dict(w_down=Q + 2), 1, b"aligned"), (dict(ids=P + 1), 1, b"aligned"),
    (dict(y=R + 0x8001), 1, b"aligned"), (dict(y=R + 0x8002, y_dtype=2), 1, b"aligned"), (dict(y=(R + 0x8000, 63)), 2, b"stride"),
    (dict(add=(R + 0x9000, 40)), 2, b"stride"), (dict(add=(R + 0x8000, 72)), 1, b"y in place of add"),
    (dict(y=Q), 1, b"operands"), (dict(y=P), 1, b"operands"),
])
def test_experts(L, kw, code, text):
    refused(L, L.tq_experts_forward(ctypes.byref(experts(**kw)), P, 1 << 30, None), code, text)


def test_experts_workspace(L):
    n = ctypes.c_size_t()
    f = L.tq_experts_workspace_size
    assert f(4, 2, 8, 64, 32, None) == 1
    for a in ((-1, 2, 8, 64, 32), (4, 0, 8, 64, 32), (4, 2, 0, 64, 32), (4, 2, 8, 60, 32), (4, 2, 8, 64, 0)):
        assert f(*a, ctypes.byref(n)) == 2
    assert f(1025, 1, 8, 64, 32, ctypes.byref(n)) == 5
    assert f(4, 2, 8, 64, 32, ctypes.byref(n)) == 0 and n.value >= 8 * 32 * 2 + 8 * 64 * 4
    d = ctypes.byref(experts())
    refused(L, L.tq_experts_forward(None, P, n.value, None), 1, b"descriptor")
    refused(L, L.tq_experts_forward(d, None, n.value, None), 1, b"ws is NULL")
    refused(L, L.tq_experts_forward(d, P + 64, n.value, None), 1, b"256")
    refused(L, L.tq_experts_forward(d, P, n.value - 1, None), 2, b"ws_bytes")
    assert L.tq_experts_forward(ctypes.byref(experts(T=0, ids=None, x=None, y=None)), None, 0, None) == 0


def test_int8_kernels_follow_from_sizes():
    from tests.int8_cases import CASES, kernel_of
    for kernel, *sizes in CASES:
        assert kernel_of(*sizes) == kernel
    kinds = {c[0] for c in CASES}
    for g in (1, 3, 60, 64, 65, 1024):
        for r in (1, 17, 300, 5000, 70000, 1 << 20):
            for i in (16, 2048, 16384):
                for o in (8, 1408, 16384):
                    assert kernel_of(g, r, i, o) in kinds


# ---- what the torch functions check ------------------------------------------------


def test_tensors_on_the_host_are_refused(L):
    import torch
    x, q, c = torch.zeros((4, 64)), torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: tq.int8_quant_rows(x, q, c), lambda: tq.int8_gemm(q, c, q, c, x), lambda: tq.swiglu(x, x[:, :32]),
                 lambda: tq.swiglu_int8(x, q, c), lambda: tq.swiglu_grad(x, x[:, :32], x), lambda: tq.combine(x, i, x),
                 lambda: tq.combine_grad(x, i, dz=x), lambda: tq.experts_forward(x, i, c, x, x, x, q)):
        with pytest.raises(tq.TileQError, match="not a tensor on a GPU"):
            call()


@pytest.fixture
def no_device(monkeypatch):
    from bit_rank_post_amd import ops
    monkeypatch.setattr(ops, "_device", lambda fn, *t: 0)

    def reached(fn, *a):
        raise AssertionError(f"{fn} would have been called")

    monkeypatch.setattr(ops, "_call", reached)


def meta(*shape, dtype="float16"):
    import torch
    return torch.empty(shape, dtype=getattr(torch, dtype), device="meta")


I8, F32, I32, U8, BF = "int8", "float32", "int32", "uint8", "bfloat16"
BIG = (1 << 32) + 4


def layer_args(T=4, k=2, E=8, d=64, ff=32, **kw):
    a = dict(x=meta(T, d), ids=meta(T, k, dtype=I32), w=meta(T, k, dtype=F32), w_up=meta(E, 2 * ff, d),
             w_down=meta(E, d, ff), y=meta(T, d), ws=meta(512, dtype=U8))
    a.update(kw)
    return a


@pytest.mark.parametrize("call,text", [
    (lambda: tq.int8_quant_rows(meta(BIG, 16), meta(BIG, 16, dtype=I8), meta(BIG, dtype=F32)), "32 bits"),
    (lambda: tq.int8_quant_rows(meta(1 << 20, 1 << 13, 16), meta(1 << 20, 1 << 13, 16, dtype=I8),
                                meta(1 << 20, 1 << 13, dtype=F32)), "32 bits"),
    (lambda: tq.int8_quant_rows(meta(4, 16), meta(4, 16), meta(4, dtype=F32)), "q is .*must be torch.int8"),
    (lambda: tq.int8_quant_rows(meta(4, 16), meta(4, 16, dtype=I8), meta(4)), "scale is .*must be torch.float32"),
    (lambda: tq.int8_quant_rows(meta(4, 16), meta(4, 32, dtype=I8), meta(4, dtype=F32)), "must be"),
    (lambda: tq.int8_quant_rows(meta(4, 16), meta(4, 16, dtype=I8), meta(5, dtype=F32)), "must be"),
    (lambda: tq.int8_quant_rows(meta(4, 16, dtype="float64"), meta(4, 16, dtype=I8), meta(4, dtype=F32)), "float16, bfloat16"),
    (lambda: tq.int8_quant_rows(meta(16), meta(16, dtype=I8), meta(1, dtype=F32)), "must be"),
    (lambda: tq.int8_quant_rows(meta(4, 32)[:, ::2], meta(4, 16, dtype=I8), meta(4, dtype=F32)), "neighbours"),
    (lambda: tq.int8_quant_rows(meta(2, 4, 32)[:, :, :16], meta(2, 4, 16, dtype=I8), meta(2, 4, dtype=F32)), "contiguous"),
    (lambda: tq.int8_gemm(meta(BIG, 16, dtype=I8), meta(BIG, dtype=F32), meta(8, 16, dtype=I8), meta(8, dtype=F32), meta(BIG, 8)), "32 bits"),
    (lambda: tq.int8_gemm(meta(4, 16), meta(4, dtype=F32), meta(8, 16, dtype=I8), meta(8, dtype=F32), meta(4, 8)), "x is"),
    (lambda: tq.int8_gemm(meta(4, 16, dtype=I8), meta(4, dtype=F32), meta(8, 16, dtype=U8), meta(8, dtype=F32), meta(4, 8)), "w is"),
    (lambda: tq.int8_gemm(meta(4, 16, dtype=I8), meta(4), meta(8, 16, dtype=I8), meta(8, dtype=F32), meta(4, 8)), "x_scale is"),
    (lambda: tq.int8_gemm(meta(4, 16, dtype=I8), meta(3, dtype=F32), meta(8, 16, dtype=I8), meta(8, dtype=F32), meta(4, 8)), "x_scale is"),
    (lambda: tq.int8_gemm(meta(4, 16, dtype=I8), meta(4, dtype=F32), meta(8, 16, dtype=I8), meta(7, dtype=F32), meta(4, 8)), "w_scale is"),
    (lambda: tq.int8_gemm(meta(4, 16, dtype=I8), meta(4, dtype=F32), meta(8, 32, dtype=I8), meta(8, dtype=F32), meta(4, 8)), "x is"),
    (lambda: tq.int8_gemm(meta(4, 16, dtype=I8), meta(4, dtype=F32), meta(2, 8, 16, dtype=I8), meta(2, 8, dtype=F32), meta(4, 8)), "off is needed"),
    (lambda: tq.int8_gemm(meta(4, 16, dtype=I8), meta(4, dtype=F32), meta(8, 16, dtype=I8), meta(8, dtype=F32), meta(5, 8)), "no src"),
    (lambda: tq.swiglu(meta(BIG, 32), meta(BIG, 16)), "32 bits"),
    (lambda: tq.swiglu(meta(4, 33), meta(4, 16)), "columns"),
    (lambda: tq.swiglu(meta(4, 32), meta(4, 32)), "h is"),
    (lambda: tq.swiglu(meta(4, 32), meta(4, 16, dtype=I8)), "float16, bfloat16"),
    (lambda: tq.swiglu(meta(4, 32), meta(4, 16), off=meta(1, dtype=I32)), "groups"),
    (lambda: tq.swiglu(meta(4, 32), meta(4, 16), off=meta(3)), "int32"),
    (lambda: tq.swiglu(meta(4, 32), meta(4, 16), off=meta(3, 1, dtype=I32)), "groups"),
    (lambda: tq.swiglu_int8(meta(4, 32), meta(4, 32, dtype=I8), meta(4, dtype=F32)), "q is"),
    (lambda: tq.swiglu_int8(meta(4, 32), meta(4, 16, dtype=I8), meta(4, 1, dtype=F32)), "scale is"),
    (lambda: tq.swiglu_grad(meta(4, 32), meta(4, 16), meta(4, 32, dtype=F32)), "da is"),
    (lambda: tq.swiglu_grad(meta(4, 32), meta(4, 16), meta(4, 16)), "da is"),
    (lambda: tq.swiglu_grad(meta(4, 32), meta(4, 16, dtype=F32), meta(4, 32), h=meta(4, 16, dtype=F32)), "h is"),
    (lambda: tq.combine(meta(8, 16), meta(BIG, dtype=I32), meta(BIG, 16)), "32 bits"),
    (lambda: tq.combine(meta(BIG, 16), meta(4, dtype=I32), meta(4, 16)), "32 bits"),
    (lambda: tq.combine(meta(8, 16), meta(7, dtype=I32), meta(4, 16)), "inv is"),
    (lambda: tq.combine(meta(8, 16), meta(8, dtype="int64"), meta(4, 16)), "int32"),
    (lambda: tq.combine(meta(8, 16), meta(2, 4, dtype=I32), meta(4, 16)), "inv is"),
    (lambda: tq.combine(meta(8, 16), meta(8, dtype=I32), meta(4, 32)), "y is"),
    (lambda: tq.combine(meta(8, 16), meta(8, dtype=I32), meta(4, 16), w=meta(4, 2)), "w is"),
    (lambda: tq.combine(meta(8, 16), meta(8, dtype=I32), meta(4, 16), w=meta(4, 3, dtype=F32)), "w is"),
    (lambda: tq.combine(meta(8, 16), meta(8, dtype=I32), meta(4, 16), add=meta(4, 16, dtype=F32)), "add is"),
    (lambda: tq.combine_grad(meta(4, 16), meta(8, dtype=I32)), "dz or dw"),
    (lambda: tq.combine_grad(meta(4, 16), meta(8, dtype=I32), dz=meta(8, 16), dw=meta(4, 2, dtype=F32)), "z for dw"),
    (lambda: tq.combine_grad(meta(4, 16), meta(8, dtype=I32), z=meta(8, 16), dz=meta(8, 16, dtype=F32)), "dz is"),
    (lambda: tq.combine_grad(meta(4, 16), meta(8, dtype=I32), z=meta(8, 16), dz=meta(9, 16)), "dz is"),
    (lambda: tq.combine_grad(meta(4, 16), meta(8, dtype=I32), z=meta(8, 24), dw=meta(4, 2, dtype=F32)), "z is"),
    (lambda: tq.experts_workspace(BIG, 2, 8, 64, 32), "32 bits"),
    (lambda: tq.experts_forward(**layer_args(T=BIG)), "32 bits"),
    (lambda: tq.experts_forward(**layer_args(x=meta(4, 64, dtype=F32))), "x is"),
    (lambda: tq.experts_forward(**layer_args(ids=meta(4, 2, dtype="int64"))), "int32"),
    (lambda: tq.experts_forward(**layer_args(ids=meta(8, dtype=I32))), "ids must"),
    (lambda: tq.experts_forward(**layer_args(w=meta(4, 3, dtype=F32))), "w is"),
    (lambda: tq.experts_forward(**layer_args(w=meta(4, 2))), "w is"),
    (lambda: tq.experts_forward(**layer_args(w_up=meta(8, 32, 64))), "w_up is"),
    (lambda: tq.experts_forward(**layer_args(w_up=meta(7, 64, 64))), "w_up is"),
    (lambda: tq.experts_forward(**layer_args(w_up=meta(8, 64, 64, dtype=BF))), "w_up is"),
    (lambda: tq.experts_forward(**layer_args(w_down=meta(8, 64, 32, dtype=I8))), "w_down is"),
    (lambda: tq.experts_forward(**layer_args(w_down=meta(8, 32, 64).transpose(1, 2))), "contiguous"),
    (lambda: tq.experts_forward(**layer_args(s_up=meta(8, 64, dtype=F32))), "go together"),
    (lambda: tq.experts_forward(**layer_args(s_up=meta(8, 64, dtype=F32), s_down=meta(8, 64, dtype=F32))), "w_up is"),
    (lambda: tq.experts_forward(**layer_args(w_up=meta(8, 64, 64, dtype=I8), w_down=meta(8, 64, 32, dtype=I8),
                                             s_up=meta(8, 32, dtype=F32), s_down=meta(8, 64, dtype=F32))), "s_up is"),
    (lambda: tq.experts_forward(**layer_args(w_up=meta(8, 64, 64, dtype=I8), w_down=meta(8, 64, 32, dtype=I8),
                                             s_up=meta(8, 64, dtype=F32), s_down=meta(8, 64))), "s_down is"),
    (lambda: tq.experts_forward(**layer_args(y=meta(4, 32))), "y is"),
    (lambda: tq.experts_forward(**layer_args(add=meta(4, 64, dtype=F32))), "add is"),
])
def test_torch_refusals(no_device, call, text):
    with pytest.raises(tq.TileQError, match=text):
        call()


@pytest.mark.parametrize("name", ["int8_quant_rows", "int8_gemm", "swiglu", "swiglu_int8", "swiglu_grad", "combine",
                                  "combine_grad", "experts_forward", "experts_workspace"])
def test_offered(name):
    from bit_rank_post_amd import ops
    assert getattr(tq, name) is getattr(ops, name)
