"""Operators around a layer of experts on torch tensors: products grouped by
expert with their gradients, products in 8-bit floating point with a scale for
each block of 128, and the norms before and after a block.

Argument marshalling and the checks that only tensors allow (shapes, strides,
dtypes, devices; the C ABI sees pointers); the work runs in the HIP kernels
behind include/tileq.h, whose comments give each operator's definition.
Outputs are caller-allocated tensors.  Calls are asynchronous on `stream` (a
torch stream or a raw handle; default: torch's current stream of the tensors'
device) and can be captured in a graph.  A refused call raises TileQError and
launches nothing.
"""
from __future__ import annotations

import ctypes

import torch

from . import (TQ_BF16, TQ_F16, TQ_F32, BlockDesc, GroupDesc, NormDesc, NormGradDesc, Rows, TileQError, _check,
               lib)

_DT = {torch.float16: TQ_F16, torch.bfloat16: TQ_BF16, torch.float32: TQ_F32}
E4M3 = torch.float8_e4m3fn
EINVAL, ESHAPE, EUNSUPPORTED = 1, 2, 5


def _ptr(t):
    return None if t is None else t.data_ptr()


def _refuse(fn, text, status=ESHAPE):
    raise TileQError("tq_" + fn, status, text)


def _device(fn, *tensors):
    """Index of the one device of all tensors that are given."""
    dev = -1
    for t in tensors:
        if t is None:
            continue
        d = t.get_device() if isinstance(t, torch.Tensor) else -1
        if d < 0:
            _refuse(fn, "an operand is not a tensor on a GPU", EINVAL)
        if d != dev:
            if dev >= 0:
                _refuse(fn, f"operands on cuda:{dev} and cuda:{d}", EINVAL)
            dev = d
    return dev


def _fits(fn, *sizes):
    """Sizes that the C ABI takes as 32-bit integers (ctypes would cut them)."""
    for n in sizes:
        if not -0x80000000 <= n <= 0x7FFFFFFF:
            _refuse(fn, f"a size of {n} does not fit 32 bits", EUNSUPPORTED)


_raw_stream = torch._C._cuda_getCurrentRawStream      # the handle alone, without a Stream object
_entries = {}


def _call(fn, dev, stream, *args):
    """Run the C entry with the tensors' device current, on `stream`."""
    entry = _entries.get(fn)
    if entry is None:
        entry = _entries[fn] = getattr(lib(), "tq_" + fn)
    if stream is None:
        stream = _raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        if getattr(stream, "device_index", dev) != dev:
            _refuse(fn, f"a stream of cuda:{stream.device_index} for operands on cuda:{dev}", EINVAL)
        stream = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        status = entry(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = entry(*args, stream)
    if status:
        _check("tq_" + fn, status)


def _float(fn, t, name):
    if t.dtype not in _DT:
        _refuse(fn, f"{name} is {t.dtype}: float16, bfloat16 or float32", EINVAL)
    return _DT[t.dtype]


def _shape(fn, t, name, *shape):
    if t.shape != shape:
        _refuse(fn, f"{name} is {tuple(t.shape)}, must be {shape}")


def _dense(fn, t, name):
    if not t.is_contiguous():
        _refuse(fn, f"{name} must be contiguous")


def _ld(fn, t, name):
    """Row stride of a matrix whose rows are dense and apart (a single row, or
    rows of one element, may have any stride in torch)."""
    if t.dim() != 2:
        _refuse(fn, f"{name} must have two dimensions, not {t.dim()}")
    rows, d = t.shape
    s0, s1 = t.stride()
    if s1 != 1 and d > 1:
        _refuse(fn, f"elements of a row of {name} must be neighbours")
    if rows <= 1:
        return d
    if s0 < d:
        _refuse(fn, f"rows of {name} overlap")
    return s0


def _int32(fn, t, name, *shape):
    if t is None:
        return
    if t.dtype is not torch.int32:
        _refuse(fn, f"{name} is {t.dtype}, must be int32", EINVAL)
    _shape(fn, t, name, *shape)
    _dense(fn, t, name)


def _group_desc(fn, groups, rows, d_in, d_out, act, off, src, src_div, x_rows, ldx, ldy):
    if off is None and groups != 1:
        _refuse(fn, f"off is needed with {groups} groups", EINVAL)
    _int32(fn, off, "off", groups + 1)
    _int32(fn, src, "src", rows)
    if src is None and x_rows != rows:
        _refuse(fn, f"x has {x_rows} rows for {rows} grouped rows and no src")
    _fits(fn, groups, rows, d_in, d_out, src_div, x_rows)
    return GroupDesc(groups, rows, d_in, d_out, act, _ptr(off), _ptr(src), src_div, x_rows, ldx, ldy)


def group_gemm(x, w, y, off=None, src=None, src_div=1, stream=None):
    """y[r] = W_g x[src[r] // src_div] for the rows off[g] .. off[g+1]-1 of each
    expert g: x [x_rows][d_in] and w [groups][d_out][d_in] float16 or bfloat16,
    y [rows][d_out] float16, bfloat16 or float32, off int32 [groups + 1] (not
    needed with one group), src int32 [rows] (without it row r of x).  w may
    also be one matrix [d_out][d_in]."""
    fn = "group_gemm"
    dev = _device(fn, x, w, y, off, src)
    w = w[None] if w.dim() == 2 else w
    if w.dim() != 3:
        _refuse(fn, "w must be [groups][d_out][d_in]")
    if x.dtype != w.dtype or x.dtype not in (torch.float16, torch.bfloat16):
        _refuse(fn, f"x is {x.dtype} and w {w.dtype}: both float16 or both bfloat16", EINVAL)
    G, d_out, d_in = w.shape
    _dense(fn, w, "w")
    ldx, ldy, ydt = _ld(fn, x, "x"), _ld(fn, y, "y"), _float(fn, y, "y")
    _shape(fn, x, "x", x.shape[0], d_in)
    _shape(fn, y, "y", y.shape[0], d_out)
    d = _group_desc(fn, G, y.shape[0], d_in, d_out, _DT[x.dtype], off, src, src_div, x.shape[0], ldx, ldy)
    _call(fn, dev, stream, ctypes.byref(d), _ptr(x), _ptr(w), _ptr(y), ydt)


def group_gemm_dx(dy, w, dx, off=None, stream=None):
    """dx[r] = W_g^T dy[r]: dy [rows][d_out] and w [groups][d_out][d_in] float16
    or bfloat16, dx [rows][d_in] float16, bfloat16 or float32.  One row per
    grouped row: rows that were gathered from the same row of x are added by
    the caller (index_add_)."""
    fn = "group_gemm_dx"
    dev = _device(fn, dy, w, dx, off)
    w = w[None] if w.dim() == 2 else w
    if w.dim() != 3:
        _refuse(fn, "w must be [groups][d_out][d_in]")
    if dy.dtype != w.dtype or dy.dtype not in (torch.float16, torch.bfloat16):
        _refuse(fn, f"dy is {dy.dtype} and w {w.dtype}: both float16 or both bfloat16", EINVAL)
    G, d_out, d_in = w.shape
    _dense(fn, w, "w")
    ldx, ldy, xdt = _ld(fn, dx, "dx"), _ld(fn, dy, "dy"), _float(fn, dx, "dx")
    _shape(fn, dy, "dy", dy.shape[0], d_out)
    _shape(fn, dx, "dx", dy.shape[0], d_in)
    d = _group_desc(fn, G, dy.shape[0], d_in, d_out, _DT[dy.dtype], off, None, 1, dy.shape[0], ldx, ldy)
    _call(fn, dev, stream, ctypes.byref(d), _ptr(dy), _ptr(w), _ptr(dx), xdt)


def group_gemm_dw(dy, x, dw, off=None, src=None, src_div=1, stream=None):
    """dw[g] = sum over the rows r of expert g of dy[r] x[src[r] // src_div]^T
    (zero for an expert without rows): dy [rows][d_out] and x [x_rows][d_in]
    float16 or bfloat16, dw [groups][d_out][d_in] float16, bfloat16 or float32."""
    fn = "group_gemm_dw"
    dev = _device(fn, dy, x, dw, off, src)
    dw = dw[None] if dw.dim() == 2 else dw
    if dw.dim() != 3:
        _refuse(fn, "dw must be [groups][d_out][d_in]")
    if dy.dtype != x.dtype or x.dtype not in (torch.float16, torch.bfloat16):
        _refuse(fn, f"dy is {dy.dtype} and x {x.dtype}: both float16 or both bfloat16", EINVAL)
    G, d_out, d_in = dw.shape
    _dense(fn, dw, "dw")
    ldx, ldy, wdt = _ld(fn, x, "x"), _ld(fn, dy, "dy"), _float(fn, dw, "dw")
    _shape(fn, x, "x", x.shape[0], d_in)
    _shape(fn, dy, "dy", dy.shape[0], d_out)
    d = _group_desc(fn, G, dy.shape[0], d_in, d_out, _DT[x.dtype], off, src, src_div, x.shape[0], ldx, ldy)
    _call(fn, dev, stream, ctypes.byref(d), _ptr(dy), _ptr(x), _ptr(dw), wdt)


def _blocks(n):
    return -(-n // 128)


def fp8_quant_rows(x, q, scale, stream=None):
    """x [rows][d] float16, bfloat16 or float32 -> q [rows][d] float8_e4m3fn with
    a scale for each 128 neighbours of a row, scale float32 [rows][ceil(d/128)]."""
    fn = "fp8_quant_rows"
    dev = _device(fn, x, q, scale)
    xdt, ldx = _float(fn, x, "x"), _ld(fn, x, "x")
    rows, d = x.shape
    _fits(fn, rows, d)
    if q.dtype != E4M3 or scale.dtype != torch.float32:
        _refuse(fn, f"q is {q.dtype} and scale {scale.dtype}: float8_e4m3fn and float32", EINVAL)
    _shape(fn, q, "q", rows, d)
    _shape(fn, scale, "scale", rows, _blocks(d))
    _dense(fn, q, "q")
    _dense(fn, scale, "scale")
    _call(fn, dev, stream, _ptr(x), xdt, rows, d, ldx, _ptr(q), _ptr(scale))


def fp8_quant_blocks(w, q, scale, stream=None):
    """w [groups][d_out][d_in] (or one matrix) float16, bfloat16 or float32 -> q
    of the same shape in float8_e4m3fn with a scale for each 128 x 128 block,
    scale float32 [groups][ceil(d_out/128)][ceil(d_in/128)]."""
    fn = "fp8_quant_blocks"
    dev = _device(fn, w, q, scale)
    wdt = _float(fn, w, "w")
    if w.dim() not in (2, 3):
        _refuse(fn, "w must be [groups][d_out][d_in]")
    if q.dtype != E4M3 or scale.dtype != torch.float32:
        _refuse(fn, f"q is {q.dtype} and scale {scale.dtype}: float8_e4m3fn and float32", EINVAL)
    _shape(fn, q, "q", *w.shape)
    o, i = w.shape[-2:]
    _fits(fn, *w.shape)
    _shape(fn, scale, "scale", *w.shape[:-2], _blocks(o), _blocks(i))
    for name, t in (("w", w), ("q", q), ("scale", scale)):
        _dense(fn, t, name)
    _call(fn, dev, stream, _ptr(w), wdt, w.shape[0] if w.dim() == 3 else 1, o, i, _ptr(q), _ptr(scale))


def fp8_gemm(x, x_scale, w, w_scale, y, off=None, src=None, src_div=1, stream=None):
    """The product of group_gemm on operands of fp8_quant_rows (x, x_scale) and
    fp8_quant_blocks (w, w_scale): y [rows][d_out] float16, bfloat16 or
    float32.  src gathers the rows of x and of x_scale alike."""
    fn = "fp8_gemm"
    dev = _device(fn, x, x_scale, w, w_scale, y, off, src)
    if w.dim() == 2:
        w, w_scale = w[None], w_scale[None]
    if w.dim() != 3:
        _refuse(fn, "w must be [groups][d_out][d_in]")
    for name, t, dt in (("x", x, E4M3), ("w", w, E4M3), ("x_scale", x_scale, torch.float32),
                        ("w_scale", w_scale, torch.float32)):
        if t.dtype != dt:
            _refuse(fn, f"{name} is {t.dtype}, must be {dt}", EINVAL)
    G, d_out, d_in = w.shape
    ldx, ldy, ydt = _ld(fn, x, "x"), _ld(fn, y, "y"), _float(fn, y, "y")
    _shape(fn, x, "x", x.shape[0], d_in)
    _shape(fn, y, "y", y.shape[0], d_out)
    _shape(fn, x_scale, "x_scale", x.shape[0], _blocks(d_in))
    _shape(fn, w_scale, "w_scale", G, _blocks(d_out), _blocks(d_in))
    for name, t in (("w", w), ("x_scale", x_scale), ("w_scale", w_scale)):
        _dense(fn, t, name)
    d = _group_desc(fn, G, y.shape[0], d_in, d_out, TQ_F16, off, src, src_div, x.shape[0], ldx, ldy)
    _call(fn, dev, stream, ctypes.byref(d), _ptr(x), _ptr(x_scale), _ptr(w), _ptr(w_scale), _ptr(y), ydt)


GATE_NONE, GATE_TOKEN, GATE_FULL = 0, 1, 2
_ABSENT = Rows(None, 0)


def _mat(fn, t, name, T, d, dtype):
    """tq_rows of an optional [T][d] tensor of one dtype."""
    if t is None:
        return _ABSENT
    if t.dtype is not dtype:
        _refuse(fn, f"{name} is {t.dtype}, must be {dtype}", EINVAL)
    if t.shape != (T, d):
        _refuse(fn, f"{name} is {tuple(t.shape)}, must be {(T, d)}")
    return Rows(t.data_ptr(), _ld(fn, t, name))


def _gate(fn, t, name, T, d, act):
    if t is None:
        return GATE_NONE, _ABSENT
    if t.dim() == 2:
        return GATE_FULL, _mat(fn, t, name, T, d, act)
    if t.dtype != torch.float32:
        _refuse(fn, f"{name} of one value per token is {t.dtype}, must be float32", EINVAL)
    _shape(fn, t, name, T)
    if T > 1 and t.stride(0) < 1:
        _refuse(fn, f"values of {name} must be apart")
    return GATE_TOKEN, Rows(t.data_ptr(), t.stride(0) if T > 1 else 1)


def _vec(fn, t, name, n, dtypes):
    if t is None:
        return
    if t.dtype not in dtypes:
        _refuse(fn, f"{name} is {t.dtype}", EINVAL)
    if t.shape != (n,):
        _refuse(fn, f"{name} is {tuple(t.shape)}, must be {(n,)}")
    if not t.is_contiguous():
        _refuse(fn, f"{name} must be contiguous")


def _weights(fn, w_post, w_next, d):
    _vec(fn, w_post, "w_post", d, _DT)
    _vec(fn, w_next, "w_next", d, _DT)
    if w_post is not None and w_next is not None and w_post.dtype != w_next.dtype:
        _refuse(fn, "w_post and w_next must have one dtype", EINVAL)
    w = w_post if w_post is not None else w_next
    return TQ_F32 if w is None else _DT[w.dtype]


def norm_residual(x, y=None, n=None, b=None, w_post=None, w_next=None, gate=None, alpha=1.0, eps=1e-6,
                  rstd_post=None, rstd_next=None, stream=None):
    """y = x + alpha * gate * p(b) with p(b) = w_post * b / rms(b) (p(b) = b
    without w_post), then n = w_next * y / rms(y).  x and y [T][d] are the
    residual stream, b [T][d] the block's output, n [T][d] the next block's
    input (dtype of b).  Only x, n and w_next: the norm before a first block;
    without n: the residual alone.  gate: float32 [T], or [T][d] of b's dtype.
    rstd_post, rstd_next (float32 [T]) take 1 / rms for norm_residual_grad.
    y may be x, and n may be b."""
    fn = "norm_residual"
    dev = _device(fn, x, y, n, b, w_post, w_next, gate, rstd_post,
                  rstd_next)
    sdt, ldx = _float(fn, x, "x"), _ld(fn, x, "x")
    T, d = x.shape
    _fits(fn, T, d)
    a = b if b is not None else n
    act = x.dtype if a is None else a.dtype
    if act not in _DT:
        _refuse(fn, f"b and n are {act}: float16, bfloat16 or float32", EINVAL)
    kind, g = _gate(fn, gate, "gate", T, d, act)
    _vec(fn, rstd_post, "rstd_post", T, (torch.float32,))
    _vec(fn, rstd_next, "rstd_next", T, (torch.float32,))
    desc = NormDesc(T, d, sdt, _DT[act], _weights(fn, w_post, w_next, d), kind, alpha, eps,
                    Rows(x.data_ptr(), ldx), _mat(fn, b, "b", T, d, act), _mat(fn, y, "y", T, d, x.dtype),
                    _mat(fn, n, "n", T, d, act), g, _ptr(w_post), _ptr(w_next), _ptr(rstd_post),
                    _ptr(rstd_next))
    _call(fn, dev, stream, ctypes.byref(desc))


def norm_residual_grad(y, dx=None, dy=None, dn=None, b=None, db=None, w_post=None, w_next=None, gate=None,
                       dgate=None, dw_post=None, dw_next=None, alpha=1.0, rstd_post=None, rstd_next=None,
                       ws=None, stream=None):
    """Gradients of norm_residual: y as it wrote it, dy (what reaches y from
    elsewhere) and dn or one of them in; dx, db, dw_post, dw_next (float32
    [d]) and dgate (as gate) out, each None when not wanted.  rstd_* as the
    forward wrote them.  ws: uint8 workspace of norm_grad_workspace(T, d)
    bytes for the weights' gradients (None: allocated by torch for the call).
    dx may be dy, and db may be dn."""
    fn = "norm_residual_grad"
    dev = _device(fn, y, dx, dy, dn, b, db, w_post, w_next, gate,
                  dgate, dw_post, dw_next, rstd_post, rstd_next,
                  ws)
    sdt = _float(fn, y, "y")
    _ld(fn, y, "y")
    T, d = y.shape
    _fits(fn, T, d)
    a = b if b is not None else dn
    act = y.dtype if a is None else a.dtype
    if act not in _DT:
        _refuse(fn, f"b and dn are {act}: float16, bfloat16 or float32", EINVAL)
    kind, g = _gate(fn, gate, "gate", T, d, act)
    dkind, dg = _gate(fn, dgate, "dgate", T, d, act)
    if dgate is not None and dkind != kind:
        _refuse(fn, "dgate must have the gate's shape", EINVAL)
    for name, t, n in (("rstd_post", rstd_post, T), ("rstd_next", rstd_next, T), ("dw_post", dw_post, d),
                       ("dw_next", dw_next, d)):
        _vec(fn, t, name, n, (torch.float32,))
    desc = NormGradDesc(T, d, sdt, _DT[act], _weights(fn, w_post, w_next, d), kind, alpha,
                        _mat(fn, y, "y", T, d, y.dtype), _mat(fn, dy, "dy", T, d, y.dtype),
                        _mat(fn, dn, "dn", T, d, act), _mat(fn, b, "b", T, d, act), g,
                        _mat(fn, dx, "dx", T, d, y.dtype), _mat(fn, db, "db", T, d, act), dg,
                        _ptr(w_post), _ptr(w_next), _ptr(rstd_post), _ptr(rstd_next), _ptr(dw_post),
                        _ptr(dw_next))
    if ws is not None:
        _dense(fn, ws, "ws")
    elif dw_post is not None or dw_next is not None:
        # allocated with the call's stream current: the pool then hands the memory
        # on in that stream's order (and keeps it, when the stream is captured)
        need = norm_grad_workspace(T, d)
        s = stream
        if s is not None and not hasattr(s, "cuda_stream"):
            s = torch.cuda.ExternalStream(s, device=dev)
        with torch.cuda.stream(s):
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _call(fn, dev, stream, ctypes.byref(desc), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size())


def norm_grad_workspace(T, d):
    """Bytes of workspace of norm_residual_grad."""
    n = ctypes.c_size_t()
    _fits("norm_grad_workspace_size", T, d)
    _check("tq_norm_grad_workspace_size", lib().tq_norm_grad_workspace_size(T, d, ctypes.byref(n)))
    return n.value


def group_slots_workspace(T, topk, K):
    """Bytes of workspace of group_slots."""
    n = ctypes.c_size_t()
    _fits("group_slots_workspace_size", T, topk, K)
    _check("tq_group_slots_workspace_size", lib().tq_group_slots_workspace_size(T, topk, K, ctypes.byref(n)))
    return n.value


def group_slots(ids, K, off, perm, inv, ws, stream=None):
    """Slots of router ids (int32 [T][topk]) grouped by expert: off int32
    [K + 1], perm int32 [T * topk] (the src of the grouped products, with
    src_div = topk), inv int32 [T * topk] (row of each slot, -1 for an id
    outside [0, K)).  ws: uint8 tensor of group_slots_workspace(T, topk, K)
    bytes; its first int32 holds the number of dropped slots afterwards.  Without
    tokens all offsets are 0."""
    fn = "group_slots"
    dev = _device(fn, ids, off, perm, inv, ws)
    if ids.dim() != 2:
        _refuse(fn, "ids must be [T][topk]")
    T, k = ids.shape
    _fits(fn, T, k, K)
    _int32(fn, ids, "ids", T, k)
    _int32(fn, off, "off", K + 1)
    _int32(fn, perm, "perm", T * k)
    _int32(fn, inv, "inv", T * k)
    _dense(fn, ws, "ws")
    _call(fn, dev, stream, _ptr(ids), T, k, K, _ptr(off), _ptr(perm), _ptr(inv), _ptr(ws),
          ws.numel() * ws.element_size())
    if T == 0:                      # the C call writes nothing then
        s = stream
        if s is not None and not hasattr(s, "cuda_stream"):
            s = torch.cuda.ExternalStream(s, device=dev)
        with torch.cuda.stream(s):
            off.zero_()
            ws.view(-1).view(torch.uint8)[:4].zero_()


def block_forward(layer, x, y, router, w_pre, topk, ids_out, gates_out, ws, w_post=None, gate=None, alpha=1.0,
                  eps=1e-6, stream=None):
    """Layer.block_forward."""
    fn = "block_forward"
    dev = _device(fn, x, y, router, w_pre, ids_out, gates_out, ws, w_post, gate)
    act = torch.float16 if layer.act == TQ_F16 else torch.bfloat16
    sdt, T, d = _float(fn, x, "x"), x.shape[0], layer.d_model
    _fits(fn, T, topk)
    for name, t in (("x", x), ("y", y)):
        _shape(fn, t, name, T, d)
        _dense(fn, t, name)
        if t.dtype is not x.dtype:
            _refuse(fn, f"{name} is {t.dtype}, must be {x.dtype}", EINVAL)
    _shape(fn, router, "router", layer.K, d)
    _dense(fn, router, "router")
    if router.dtype is not act:
        _refuse(fn, f"router is {router.dtype}, must be {act}", EINVAL)
    if w_pre is None:
        _refuse(fn, "w_pre is needed", EINVAL)
    _int32(fn, ids_out, "ids_out", T, topk)
    _shape(fn, gates_out, "gates_out", T, topk)
    _dense(fn, gates_out, "gates_out")
    _dense(fn, ws, "ws")
    if gates_out.dtype is not torch.float32:
        _refuse(fn, f"gates_out is {gates_out.dtype}, must be float32", EINVAL)
    kind, g = _gate(fn, gate, "gate", T, d, act)
    desc = BlockDesc(topk, sdt, _weights(fn, w_post, w_pre, d), kind, alpha, eps, _ptr(w_pre), _ptr(w_post),
                     _ptr(router), g)
    _call(fn, dev, stream, layer.h, ctypes.byref(desc), _ptr(x), T, _ptr(ids_out), _ptr(gates_out), _ptr(y),
          _ptr(ws), ws.numel() * ws.element_size())
