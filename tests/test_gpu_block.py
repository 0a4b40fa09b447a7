"""The operators together: a block around a packed layer (norm, router, layer,
norm, gate, residual), experts that are not packed from router logits to the
gradients of their weights, and the grouping of router ids."""
import numpy as np
import pytest
import torch

import bit_rank_post_amd as tq
import synth
from bit_rank_post_amd import io as tqio
from bit_rank_post_amd import ops
from oracle import tileq_ref
from tests.gpu_util import need_gpu
from tests.ops_util import DT, check, gen, half_step, normal
from tests.test_gpu_parity import small_swiglu

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# ---- grouping ----------------------------------------------------------------


@pytest.mark.parametrize("T,k,K", [(1, 1, 1), (1, 2, 8), (3, 4, 60), (64, 6, 64), (1024, 4, 60), (1025, 2, 8),
                                   (5000, 6, 64), (4097, 32, 256), (30000, 1, 3)])
@pytest.mark.parametrize("bad", [False, True])
def test_group_slots(T, k, K, bad):
    print(f"[case] slots {T} {k} {K} {bad}", flush=True)
    rng = np.random.default_rng(T + k)
    ids = rng.integers(0, K, (T, k)).astype(np.int32)
    if bad:
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = K
    S = T * k
    off, perm, inv = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (K + 1, S, S))
    ws = torch.full((ops.group_slots_workspace(T, k, K),), 255, dtype=torch.uint8, device="cuda")
    tq.group_slots(torch.from_numpy(ids).cuda(), K, off, perm, inv, ws)
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < K)
    slots = np.nonzero(ok)[0]
    want = slots[np.argsort(flat[slots], kind="stable")]
    woff = np.concatenate([[0], np.cumsum(np.bincount(flat[slots], minlength=K))])
    winv = np.full(S, -1)
    winv[want] = np.arange(len(want))
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(perm.cpu().numpy()[:len(want)], want)
    assert np.array_equal(inv.cpu().numpy(), winv)
    assert int(ws[:4].view(torch.int32).item()) == S - len(want)


# ---- experts that are not packed ---------------------------------------------


class Experts:
    """K SwiGLU experts in 16 bits, top-k routing from logits: the operators of
    the package with torch's elementwise operations between them."""

    def __init__(self, K, d, ff, dt, seed):
        g = gen(seed)
        self.K, self.dt = K, dt
        self.gate_up = normal(g, (K, 2 * ff, d), d ** -0.5, dt).cuda()
        self.down = normal(g, (K, d, ff), ff ** -0.5, dt).cuda()

    def forward(self, x, logits, k, out):
        T, d = x.shape
        self.x, self.k = x, k
        ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
        self.w = torch.empty((T, k), device="cuda")
        tq.router_topk(logits, k, ids, self.w)
        S, ff = T * k, self.down.shape[2]
        self.off, self.perm, self.inv = (torch.empty(n, dtype=torch.int32, device="cuda")
                                         for n in (self.K + 1, S, S))
        ws = torch.empty(ops.group_slots_workspace(T, k, self.K), dtype=torch.uint8, device="cuda")
        tq.group_slots(ids, self.K, self.off, self.perm, self.inv, ws)
        self.a = torch.empty((S, 2 * ff), dtype=self.dt, device="cuda")
        tq.group_gemm(x, self.gate_up, self.a, off=self.off, src=self.perm, src_div=k)
        gate, up = self.a.float().chunk(2, dim=1)
        self.h = (torch.nn.functional.silu(gate) * up).to(self.dt)
        o = torch.empty((S, d), dtype=torch.float32, device="cuda")
        tq.group_gemm(self.h, self.down, o, off=self.off)
        out.copy_((o[self.inv.long()].view(T, k, d) * self.w[:, :, None]).sum(1))
        return ids

    def backward(self, dout):
        """Gradients of x, gate_up and down for that of out."""
        T, d = self.x.shape
        tok = (self.perm // self.k).long()
        do = (dout.float()[tok] * self.w.reshape(-1)[self.perm.long()][:, None]).to(self.dt)
        dh = torch.empty(self.h.shape, device="cuda")
        tq.group_gemm_dx(do, self.down, dh, off=self.off)
        d_down = torch.empty(self.down.shape, device="cuda")
        tq.group_gemm_dw(do, self.h, d_down, off=self.off)
        gate, up = self.a.float().chunk(2, dim=1)
        s = torch.sigmoid(gate)
        da = torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], dim=1).to(self.dt)
        dxr = torch.empty((len(tok), d), device="cuda")
        tq.group_gemm_dx(da, self.gate_up, dxr, off=self.off)
        d_gu = torch.empty(self.gate_up.shape, device="cuda")
        tq.group_gemm_dw(da, self.x, d_gu, off=self.off, src=self.perm, src_div=self.k)
        return torch.zeros((T, d), device="cuda").index_add_(0, tok, dxr), d_gu, d_down


def experts_ref(x, gate_up, down, ids, w):
    y = torch.zeros_like(x)
    for e in range(gate_up.shape[0]):
        for j in range(ids.shape[1]):
            t = (ids[:, j] == e).nonzero()[:, 0]
            if len(t):
                gate, up = (x[t] @ gate_up[e].t()).chunk(2, dim=1)
                y = y.index_add(0, t, (torch.nn.functional.silu(gate) * up @ down[e].t()) * w[t, j, None])
    return y


@pytest.mark.parametrize("T,K,k,d,ff,dtype", [(1, 8, 2, 128, 64, "f16"), (5, 60, 4, 256, 96, "bf16"),
                                              (300, 8, 2, 256, 136, "f16"), (700, 16, 3, 136, 264, "bf16")])
def test_experts_from_logits_to_gradients(T, K, k, d, ff, dtype):
    print(f"[case] experts {T} {K} {k} {d} {ff} {dtype}", flush=True)
    dt = DT[dtype]
    E = Experts(K, d, ff, dt, 1)
    g = gen(2)
    x, logits, dout = normal(g, (T, d), 1.0, dt).cuda(), torch.randn((T, K), generator=g).cuda(), normal(
        g, (T, d), 1.0, torch.float32).cuda()
    out = torch.empty((T, d), device="cuda")
    ids = E.forward(x, logits, k, out)
    grads = E.backward(dout)
    p = [t.double().cpu().requires_grad_() for t in (x, E.gate_up, E.down)]
    ref = experts_ref(*p, ids.cpu().long(), E.w.double().cpu())
    ref.backward(dout.double().cpu())
    # Rounded to 16 bits on the way: a and h forward (what is read of them then
    # carries u = eps/2 of the value); do, da backward.  Forward: each term of
    # out is off by u (|a| derivative) + u; with |silu'| <= 1.1 and |silu(v)|
    # <= |v| that is at most 3.1 u of the sum of magnitudes.  Backward, da has
    # the errors of do, a (through the second derivative, < 0.5 |up| |a|) and
    # its own: 5 u of magnitudes.  f32 sums are far below.
    u = torch.finfo(dt).eps / 2
    with torch.no_grad():
        xa, gu, dn = p[0].abs(), p[1].abs(), p[2].abs()
        wabs = E.w.double().cpu()
        mag_out, mag = torch.zeros_like(ref), [torch.zeros_like(t) for t in p]
        for e in range(K):
            for j in range(k):
                t = (ids.cpu()[:, j] == e).nonzero()[:, 0]
                if not len(t):
                    continue
                A = xa[t] @ gu[e].t()                              # magnitudes of a, without cancellation
                Ag, Au = A.chunk(2, dim=1)
                H = Ag * Au
                mag_out.index_add_(0, t, (H @ dn[e].t()) * wabs[t, j, None])
                D = dout.double().cpu().abs()[t] * wabs[t, j, None]
                dH = D @ dn[e]
                dA = torch.cat([dH * Au * (1.1 + 0.5 * Ag), dH * Ag], dim=1)
                mag[0].index_add_(0, t, dA @ gu[e])
                mag[1][e] += dA.t() @ xa[t]
                mag[2][e] += D.t() @ H
    check("out", out, ref.detach(), 3.1 * 1.01 * u * mag_out + 1e-6 * mag_out)
    for name, got, t, m in zip(("dx", "d gate_up", "d down"), grads, p, mag):
        check(name, got, t.grad, 5 * 1.01 * u * m + 1e-6 * m)


# ---- the block around a packed layer -----------------------------------------


def block_inputs(L, T, sdt, gate, seed):
    g = gen(seed)
    d, act = L.d_model, DT["f16" if L.act == tq.TQ_F16 else "bf16"]
    x = normal(g, (T, d), 1.5, DT[sdt])
    w_pre, w_post = (1 + normal(g, (d,), 0.1, torch.float32) for _ in range(2))
    router = normal(g, (L.K, d), d ** -0.5, act)
    gv = None
    if gate == "token":
        gv = torch.sigmoid(normal(g, (T,), 1.0, torch.float32))
    elif gate == "full":
        gv = torch.sigmoid(normal(g, (T, d), 1.0, torch.float32)).to(act)
    return x, w_pre, w_post, router, gv


@pytest.mark.parametrize("act,sdt,T,gate,post", [
    ("f16", "f16", 1, "none", True), ("f16", "f32", 24, "token", True), ("f16", "f16", 300, "full", True),
    ("bf16", "bf16", 33, "token", True), ("bf16", "f32", 260, "none", False), ("f16", "f32", 5, "token", False)])
def test_block_forward(act, sdt, T, gate, post):
    print(f"[case] block {act} {sdt} {T} {gate} {post}", flush=True)
    layer = small_swiglu(act, 3)
    L = tqio.upload_layer(layer)
    k, d, alpha = 2, L.d_model, 0.5
    x, w_pre, w_post, router, gv = block_inputs(L, T, sdt, gate, 7)
    c = [None if t is None else t.cuda() for t in (x, w_pre, w_post, router, gv)]
    ids, gates = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    ws = torch.full((L.block_workspace_size(T, k),), 255, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(c[0])
    kw = dict(w_post=c[2] if post else None, gate=c[4], alpha=alpha)
    L.block_forward(c[0], y, c[3], c[1], k, ids, gates, ws, **kw)
    torch.cuda.synchronize()
    # the same as its four steps, bit for bit
    adt = router.dtype
    n, b = torch.empty((T, d), dtype=adt, device="cuda"), torch.empty((T, d), dtype=adt, device="cuda")
    logits = torch.empty((T, L.K), device="cuda")
    ids2, gates2, y2 = torch.empty_like(ids), torch.empty_like(gates), torch.empty_like(y)
    tq.norm_residual(c[0], n=n, w_next=c[1])
    tq.group_gemm(n, c[3], logits)
    L.forward_from_logits(n, T, logits, k, ids2, gates2, b, L.act, tqio.workspace(L, T, k))
    tq.norm_residual(c[0], y=y2, b=b, **kw)
    assert torch.equal(ids, ids2) and torch.equal(gates, gates2) and torch.equal(y, y2)
    # y in place of x
    xi = c[0].clone()
    L.block_forward(xi, xi, c[3], c[1], k, ids2, gates2, ws, **kw)
    assert torch.equal(xi, y)
    # against the definition: the layer by its oracle (within 2e-3 of the
    # largest output, its tests' bound) on the n that the block computed
    nh = n.cpu()
    nn = nh.numpy() if act == "f16" else nh.view(torch.int16).numpy().view(np.uint16)
    bref = torch.from_numpy(tileq_ref.forward(layer, nn, ids.cpu().numpy(), gates.cpu().numpy()))
    tolb = 2e-3 * bref.abs().max() + half_step(bref, adt)
    r1 = (bref.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    w = w_post.double() if post else 1.0
    g = 1.0 if gv is None else gv.double().view(T, -1)
    if post:
        # r1 moves by at most the relative error of rms(b)
        rel = (tolb.pow(2).mean(1, keepdim=True)).sqrt() * r1
        ref, dp = bref * r1 * w, r1 * w * (tolb + bref.abs() * rel) * (1 + rel)
    else:
        ref, dp = bref, tolb
    ref = x.double() + alpha * g * ref
    check("y", y, ref, alpha * g * dp * 1.01 + half_step(ref, y.dtype) + 2.0 ** -20 * ref.abs())
    L.close()


def test_block_replays_in_a_graph():
    L = tqio.upload_layer(small_swiglu("f16", 3))
    T, k = 24, 2
    x, w_pre, w_post, router, gv = [None if t is None else t.cuda() for t in block_inputs(L, T, "f16", "token", 9)]
    ids, gates = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    ws = torch.empty(L.block_workspace_size(T, k), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)

    def step():
        L.block_forward(x, y, router, w_pre, k, ids, gates, ws, w_post=w_post, gate=gv)

    step()
    torch.cuda.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        y.fill_(float("nan"))
        ws.fill_(255)
        torch.randn(1000, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    L.close()


def test_refusals():
    L = tqio.upload_layer(small_swiglu("f16", 3))
    T, k, d = 4, 2, L.d_model
    x, w_pre, w_post, router, gv = [t.cuda() for t in block_inputs(L, T, "f16", "token", 9)]
    ids, gates = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    ws = torch.empty(L.block_workspace_size(T, k), dtype=torch.uint8, device="cuda")
    y = torch.full_like(x, 3.0)

    def refused(text, *a, **kw):
        with pytest.raises(tq.TileQError, match=text):
            L.block_forward(*a, **kw)

    refused("ws_bytes", x, y, router, w_pre, k, ids, gates, ws[:-256])
    refused("not 256-byte", x, y, router, w_pre, k, ids, gates, torch.empty(ws.numel() + 64, dtype=torch.uint8,
                                                                            device="cuda")[64:])
    refused("router is", x, y, router.float(), w_pre, k, ids, gates, ws)
    refused("router is", x, y, router[:-1], w_pre, k, ids, gates, ws)
    refused("y is", x, y.float(), router, w_pre, k, ids, gates, ws)
    refused("w_pre is needed", x, y, router, None, k, ids, gates, ws)
    refused("one dtype", x, y, router, w_pre, k, ids, gates, ws, w_post=w_post.half())
    refused("ids_out", x, y, router, w_pre, k, ids.long(), gates, ws)
    refused("topk", x, y, router, w_pre, 0, torch.empty((T, 0), dtype=torch.int32, device="cuda"), torch.empty((T, 0), device="cuda"), ws)
    refused("eps", x, y, router, w_pre, k, ids, gates, ws, eps=-1.0)
    refused("contiguous", x[:, ::2].repeat(1, 2)[:, :d].t().contiguous().t(), y, router, w_pre, k, ids, gates, ws)
    torch.cuda.synchronize()
    assert (y == 3).all()
    h, dx = x.clone(), x.clone()
    for text, call in (
            ("w must be", lambda: tq.group_gemm(x, x[0], y)),
            ("both float16", lambda: tq.group_gemm(x.float(), router[None].float(), y)),
            ("off is needed", lambda: tq.group_gemm(x, torch.stack([router, router]), torch.empty((T, L.K), device="cuda"))),
            ("no src", lambda: tq.group_gemm(x, router, torch.empty((T + 1, L.K), device="cuda"))),
            ("must be", lambda: tq.group_gemm(x, router, torch.empty((T, L.K + 1), device="cuda"))),
            ("int32", lambda: tq.group_gemm(x, router, torch.empty((T, L.K), device="cuda"), off=torch.zeros(2, device="cuda"))),
            ("neighbours", lambda: tq.group_gemm(x.t().contiguous().t(), router, torch.empty((T, L.K), device="cuda"))),
            ("contiguous", lambda: tq.group_gemm(x, router[:, :64].expand(L.K, 64), torch.empty((T, L.K), device="cuda"))),
            ("overlap", lambda: tq.norm_residual(x[:1].expand(T, d), n=h, w_next=w_pre)),
            ("not a tensor", lambda: tq.norm_residual(x, n=h.cpu(), w_next=w_pre)),
            ("go together", lambda: tq.norm_residual(x, y=y, n=h, w_next=w_pre)),
            ("gate", lambda: tq.norm_residual(x, y=y, b=h, gate=torch.ones(T, device="cuda").half())),
            ("gate's shape", lambda: tq.norm_residual_grad(x, dy=h, dx=dx, b=h, gate=gv, dgate=h.clone())),
            ("must be", lambda: tq.fp8_quant_rows(x, h.to(torch.float8_e4m3fn), torch.empty((T, 1), device="cuda"))),
            ("float8", lambda: tq.fp8_quant_rows(x, h, torch.empty((T, d // 128), device="cuda"))),
            ("ids must", lambda: tq.group_slots(ids.view(-1), 8, ids, ids, ids, ws))):
        with pytest.raises(tq.TileQError, match=text):
            call()
    L.close()
