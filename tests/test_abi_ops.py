"""Refusals of the operators around a layer, on the CPU: every check runs on
the host before any launch (the pointers passed here are never dereferenced)."""
import ctypes
import os

import pytest

import bit_rank_post_amd as tq

P = 0x10000       # an aligned address, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(tq.LIB_PATH):
        pytest.skip("libtileq.so not built")
    return tq.lib()


def group(**kw):
    d = dict(groups=2, rows=64, d_in=128, d_out=64, act=tq.TQ_F16, off=P, src=None, src_div=1, x_rows=64,
             ldx=0, ldy=0)
    d.update(kw)
    return tq.GroupDesc(*[d[n] for n, _ in tq.GroupDesc._fields_])


GROUP_BAD = [
    (dict(groups=0), 2, b"groups = 0"), (dict(groups=1025), 2, b"groups = 1025"),
    (dict(groups=-3), 2, b"groups"), (dict(rows=-1), 2, b"rows = -1"), (dict(off=None), 1, b"off is NULL"),
    (dict(d_in=0), 2, b"d_in"), (dict(d_in=-128), 2, b"d_in"), (dict(d_out=0), 2, b"d_out"),
    (dict(ldx=120), 2, b"ldx"), (dict(ldy=56), 2, b"ldy"), (dict(ldx=-8), 2, b"ldx"),
    (dict(ldx=(1 << 21) + 16), 5, b"stride"),
]


@pytest.mark.parametrize("kw,code,text", GROUP_BAD)
def test_group_descriptor(L, kw, code, text):
    d = ctypes.byref(group(**kw))
    for st in (L.tq_group_gemm(d, P, P, P, 0, None), L.tq_group_gemm_dx(d, P, P, P, 0, None),
               L.tq_group_gemm_dw(d, P, P, P, 0, None), L.tq_fp8_gemm(d, P, P, P, P, P, 0, None)):
        assert st == code, L.tq_last_error()
        assert text in L.tq_last_error(), L.tq_last_error()


@pytest.mark.parametrize("kw,code,text", [
    (dict(act=tq.TQ_F32), 1, b"act"), (dict(act=7), 1, b"act"), (dict(d_in=132), 2, b"d_in"),
])
def test_group_16_bit(L, kw, code, text):
    d = ctypes.byref(group(**kw))
    for st in (L.tq_group_gemm(d, P, P, P, 0, None), L.tq_group_gemm_dx(d, P, P, P, 0, None),
               L.tq_group_gemm_dw(d, P, P, P, 0, None)):
        assert st == code and text in L.tq_last_error(), L.tq_last_error()


def test_group_pointers_types_and_sources(L):
    ok = group()
    d = ctypes.byref(ok)
    assert L.tq_group_gemm(None, P, P, P, 0, None) == 1
    assert L.tq_group_gemm(d, P, P, P, 3, None) == 1 and b"output dtype" in L.tq_last_error()
    for args in ((None, P, P), (P, None, P), (P, P, None)):
        assert L.tq_group_gemm(d, *args, 0, None) == 1 and b"NULL" in L.tq_last_error()
        assert L.tq_group_gemm_dx(d, *args, 0, None) == 1 and b"NULL" in L.tq_last_error()
        assert L.tq_group_gemm_dw(d, *args, 0, None) == 1 and b"NULL" in L.tq_last_error()
    for args in ((P + 8, P, P), (P, P + 2, P)):
        assert L.tq_group_gemm(d, *args, 0, None) == 1 and b"aligned" in L.tq_last_error()
        assert L.tq_group_gemm_dx(d, *args, 0, None) == 1 and b"aligned" in L.tq_last_error()
        assert L.tq_group_gemm_dw(d, *args, 0, None) == 1 and b"aligned" in L.tq_last_error()
    for i in (0, 1):
        args = [P + 4096, P + 8192, P]
        args[i] = P                                                   # the output in place of an operand
        assert L.tq_group_gemm(d, *args, 0, None) == 1 and b"operands" in L.tq_last_error()
        assert L.tq_group_gemm_dx(d, *args, 0, None) == 1 and b"operands" in L.tq_last_error()
        assert L.tq_group_gemm_dw(d, *args, 0, None) == 1 and b"operands" in L.tq_last_error()
        f8 = [args[0], P + 64, args[1], P + 64, P]
        assert L.tq_fp8_gemm(d, *f8, 0, None) == 1 and b"operands" in L.tq_last_error()
    # the gradients read rows of dy
    for kw in (dict(d_out=60), dict(ldy=68)):
        b = ctypes.byref(group(**kw))
        assert L.tq_group_gemm_dx(b, P, P, P, 0, None) == 2 and L.tq_group_gemm_dw(b, P, P, P, 0, None) == 2
    b = ctypes.byref(group(ldx=132))
    assert L.tq_group_gemm(b, P, P, P, 0, None) == 2 and L.tq_group_gemm_dw(b, P, P, P, 0, None) == 2
    # sources
    assert L.tq_group_gemm_dx(ctypes.byref(group(src=P)), P, P, P, 0, None) == 1
    for kw, code in ((dict(src_div=0), 2), (dict(src_div=-2), 2), (dict(x_rows=-1), 2),
                     (dict(x_rows=1 << 23), 5)):
        b = ctypes.byref(group(src=P, **kw))
        assert L.tq_group_gemm(b, P, P, P, 0, None) == code, L.tq_last_error()
        assert L.tq_group_gemm_dw(b, P, P, P, 0, None) == code, L.tq_last_error()
    # more workgroups than a launch takes
    assert L.tq_group_gemm(ctypes.byref(group(rows=2 ** 31 - 1)), P, P, P, 0, None) == 5
    big = ctypes.byref(group(groups=1, rows=1 << 30, d_in=8, d_out=1 << 20, ldy=1 << 20))
    assert L.tq_group_gemm(big, P, P + 4096, P + 8192, 0, None) == 5 and b"launch" in L.tq_last_error()


def test_no_rows_is_no_work(L):
    d = ctypes.byref(group(rows=0))
    assert L.tq_group_gemm(d, None, None, None, 0, None) == 0
    assert L.tq_group_gemm_dx(d, None, None, None, 0, None) == 0
    assert L.tq_group_gemm_dw(d, None, None, None, 0, None) == 1      # dw is still written
    assert L.tq_fp8_gemm(d, None, None, None, None, None, 0, None) == 0
    assert L.tq_fp8_quant_rows(None, 0, 0, 128, 0, None, None, None) == 0
    assert L.tq_norm_residual(ctypes.byref(norm(T=0)), None) == 0


def test_fp8(L):
    ok = ctypes.byref(group(act=99))                                  # act is not read
    assert L.tq_fp8_gemm(ok, None, P, P, P, P, 0, None) == 1 and b"NULL" in L.tq_last_error()
    for i in range(5):
        args = [P] * 5
        args[i] = None
        assert L.tq_fp8_gemm(ok, *args, 0, None) == 1, i
    for i, off in ((0, 8), (1, 2), (2, 8), (3, 1)):
        args = [P] * 5
        args[i] = P + off
        assert L.tq_fp8_gemm(ok, *args, 0, None) == 1 and b"aligned" in L.tq_last_error()
    assert L.tq_fp8_gemm(ctypes.byref(group(d_in=136)), P, P, P, P, P, 0, None) == 2
    assert L.tq_fp8_gemm(ctypes.byref(group(ldx=136)), P, P, P, P, P, 0, None) == 2
    for args, code in (((P, 3, 4, 128, 0, P, P), 1), ((P, 0, -1, 128, 0, P, P), 2), ((P, 0, 4, 120, 0, P, P), 2),
                       ((P, 0, 4, 0, 0, P, P), 2), ((P, 0, 4, 128, 100, P, P), 2), ((P, 0, 4, 128, 132, P, P), 2),
                       ((P, 2, 4, 128, 130, P, P), 2), ((None, 0, 4, 128, 0, P, P), 1), ((P, 0, 4, 128, 0, None, P), 1),
                       ((P, 0, 4, 128, 0, P, None), 1), ((P + 2, 0, 4, 128, 0, P, P), 1), ((P, 0, 4, 128, 0, P + 1, P), 1),
                       ((P, 0, 2 ** 31 - 1, 1 << 20, 0, P, P), 5)):
        assert L.tq_fp8_quant_rows(*args, None) == code, (args, L.tq_last_error())
    for args, code in (((P, 9, 1, 8, 128, P, P), 1), ((P, 0, 0, 8, 128, P, P), 2), ((P, 0, 1, 0, 128, P, P), 2),
                       ((P, 0, 1, 8, 100, P, P), 2), ((None, 0, 1, 8, 128, P, P), 1), ((P, 0, 1, 8, 128, P, None), 1),
                       ((P + 4, 0, 1, 8, 128, P, P), 1), ((P, 0, 1 << 20, 1 << 20, 1 << 20, P, P), 5)):
        assert L.tq_fp8_quant_blocks(*args, None) == code, (args, L.tq_last_error())


def norm(**kw):
    d = dict(T=4, d=64, stream_dtype=0, act=0, w_dtype=0, gate=0, alpha=1.0, eps=1e-6, x=P, b=P, y=P, n=P,
             gate_v=None, w_post=P, w_next=P, rstd_post=None, rstd_next=None)
    d.update(kw)
    vals = []
    for name, typ in tq.NormDesc._fields_:
        v = d[name]
        if typ is tq.Rows:
            v = tq.Rows(*v) if isinstance(v, tuple) else tq.Rows(v, 0)
        vals.append(v)
    return tq.NormDesc(*vals)


@pytest.mark.parametrize("kw,code,text", [
    (dict(T=-1), 2, b"T = -1"), (dict(T=1 << 22), 5, b"2^22"), (dict(d=0), 2, b"d = 0"), (dict(d=12), 2, b"d = 12"),
    (dict(d=16392), 2, b"d = 16392"), (dict(stream_dtype=3), 1, b"dtype"), (dict(act=-1), 1, b"dtype"),
    (dict(w_dtype=4), 1, b"dtype"), (dict(gate=3), 1, b"gate kind"), (dict(alpha=float("nan")), 1, b"alpha"),
    (dict(eps=-1.0), 1, b"eps"), (dict(eps=float("inf")), 1, b"eps"), (dict(x=None), 1, b"x is NULL"),
    (dict(y=None), 1, b"go together"), (dict(b=None), 1, b"go together"),
    (dict(b=None, y=None, n=None, w_post=None), 1, b"neither"), (dict(b=None, y=None), 1, b"need b"),
    (dict(b=None, y=None, w_post=None, gate=1, gate_v=P), 1, b"need b"), (dict(w_next=None), 1, b"w_next"),
    (dict(w_post=None, rstd_post=P), 1, b"rstd_post"), (dict(n=None, rstd_next=P), 1, b"rstd_next"),
    (dict(gate=1), 1, b"gate is NULL"), (dict(gate=2), 1, b"gate is NULL"), (dict(gate=1, gate_v=(P, -1)), 2, b"gate"),
    (dict(gate=1, gate_v=P + 2), 1, b"gate"), (dict(gate=2, gate_v=(P, 60)), 2, b"gate"),
    (dict(x=(P, 56)), 2, b"row stride 56 of x"), (dict(y=(P, 68)), 2, b"of y"), (dict(b=(P, 0x7001)), 2, b"of b"),
    (dict(n=P + 8), 1, b"n not 16"), (dict(x=P + 2), 1, b"x not 16"), (dict(w_post=P + 4), 1, b"w_post"),
    (dict(w_next=P + 8), 1, b"w_next"), (dict(rstd_next=P + 1), 1, b"rstd"),
    (dict(stream_dtype=2, x=(P, 66)), 2, b"of x"),
])
def test_norm(L, kw, code, text):
    assert L.tq_norm_residual(ctypes.byref(norm(**kw)), None) == code, L.tq_last_error()
    assert text in L.tq_last_error(), L.tq_last_error()


def grad(**kw):
    d = dict(T=4, d=64, stream_dtype=0, act=0, w_dtype=0, gate=0, alpha=1.0, y=P, dy=P, dn=P, b=P, gate_v=None,
             dx=P, db=P, dgate=None, w_post=P, w_next=P, rstd_post=P, rstd_next=P, dw_post=P, dw_next=P)
    d.update(kw)
    vals = []
    for name, typ in tq.NormGradDesc._fields_:
        v = d[name]
        if typ is tq.Rows:
            v = tq.Rows(*v) if isinstance(v, tuple) else tq.Rows(v, 0)
        vals.append(v)
    return tq.NormGradDesc(*vals)


@pytest.mark.parametrize("kw,code,text", [
    (dict(T=-2), 2, b"T = -2"), (dict(d=20), 2, b"d = 20"), (dict(gate=-1), 1, b"gate"), (dict(act=5), 1, b"dtype"),
    (dict(alpha=float("inf")), 1, b"alpha"), (dict(dy=None, dn=None), 1, b"neither"), (dict(y=None), 1, b"dn needs"),
    (dict(w_next=None), 1, b"dn needs"), (dict(rstd_next=None), 1, b"dn needs"), (dict(b=None), 1, b"need b"),
    (dict(rstd_post=None), 1, b"rstd_post"), (dict(w_post=None), 1, b"dw_post needs"), (dict(dn=None), 1, b"dw_next needs"),
    (dict(dgate=P), 1, b"dgate needs"), (dict(gate=1), 1, b"gate is NULL"), (dict(gate=2, gate_v=P, dgate=(P, 60)), 2, b"dgate"),
    (dict(dx=(P, 60)), 2, b"dx"), (dict(db=P + 2), 1, b"db"), (dict(dy=(P, 63)), 2, b"dy"), (dict(dn=P + 8), 1, b"dn"),
    (dict(w_post=P + 2), 1, b"w_post"), (dict(dw_next=P + 2), 1, b"dw_next"),
])
def test_norm_gradient(L, kw, code, text):
    assert L.tq_norm_residual_grad(ctypes.byref(grad(**kw)), P, 1 << 30, None) == code, L.tq_last_error()
    assert text in L.tq_last_error(), L.tq_last_error()


def test_norm_gradient_workspace(L):
    n = ctypes.c_size_t()
    assert L.tq_norm_grad_workspace_size(4, 64, None) == 1
    assert L.tq_norm_grad_workspace_size(-4, 64, ctypes.byref(n)) == 2
    assert L.tq_norm_grad_workspace_size(4, 64, ctypes.byref(n)) == 0 and n.value >= 2 * 64 * 4
    d = ctypes.byref(grad())
    assert L.tq_norm_residual_grad(d, None, 0, None) == 1
    assert L.tq_norm_residual_grad(d, P + 64, 1 << 20, None) == 1
    assert L.tq_norm_residual_grad(d, P, n.value - 1, None) == 2
    assert L.tq_norm_residual_grad(None, P, 1 << 20, None) == 1


def test_tensors_on_the_host_are_refused(L):
    import torch
    x, w, y = torch.zeros((4, 64), dtype=torch.float16), torch.zeros((1, 32, 64), dtype=torch.float16), torch.zeros((4, 32))
    for call in (lambda: tq.group_gemm(x, w, y), lambda: tq.group_gemm_dx(y.half(), w, x),
                 lambda: tq.group_gemm_dw(y.half(), x, w), lambda: tq.norm_residual(x, n=x, w_next=x[0]),
                 lambda: tq.fp8_quant_rows(x, x.to(torch.float8_e4m3fn), torch.zeros((4, 1)))):
        with pytest.raises(tq.TileQError, match="not a tensor on a GPU"):
            call()


@pytest.mark.parametrize("T,k,K,code", [(-1, 2, 8, 2), (4, 0, 8, 2), (4, 33, 64, 2), (4, 2, 0, 2), (4, 2, 257, 2),
                                        (1 << 20, 2, 8, 2), (0, 2, 8, 0), (4, 2, 256, 0)])
def test_group_slots(L, T, k, K, code):
    n = ctypes.c_size_t()
    assert L.tq_group_slots_workspace_size(T, k, K, ctypes.byref(n)) == code, L.tq_last_error()
    assert L.tq_group_slots_workspace_size(T, k, K, None) == 1
    if code or T == 0:
        assert L.tq_group_slots(P, T, k, K, P, P, P, P, 1 << 30, None) == code
        return
    assert L.tq_group_slots(P, T, k, K, P, P, P, P, n.value - 1, None) == 2
    assert L.tq_group_slots(P, T, k, K, P, P, P, P + 64, n.value, None) == 1
    for i in range(4):
        a = [P] * 5
        a[i] = None
        assert L.tq_group_slots(a[0], T, k, K, a[1], a[2], a[3], a[4], n.value, None) == 1


def test_block_without_uploads(L):
    n, h = ctypes.c_size_t(), ctypes.c_void_p()
    assert L.tq_block_workspace_size(None, 4, 2, ctypes.byref(n)) == 1
    d = tq.BlockDesc(2, 0, 0, 0, 1.0, 1e-6, P, P, P, tq.Rows(None, 0))
    assert L.tq_block_forward(None, ctypes.byref(d), P, 4, P, P, P, P, 1 << 30, None) == 1
    assert L.tq_layer_create(1, 0, 256, 512, 8, ctypes.byref(h)) == 0
    assert L.tq_block_workspace_size(h, 4, 2, ctypes.byref(n)) == 6
    assert L.tq_block_forward(h, ctypes.byref(d), P, 4, P, P, P, P, 1 << 30, None) == 6
    assert L.tq_layer_destroy(h) == 0
