"""The sum over a token's slots and its gradient, against the formulas in 64
bits.  A sum of k products in f32 by fma, one more addition for add: (k + 1) 2^-24
of the sum of magnitudes, rounded once.  A dot product of d values: at most 2^-24
of the magnitudes for each of the additions on one path, d / 64 in a lane and 6
across."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import DT, check, gen, half_step, normal

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def make(T, k, d, zdt, ydt, seed, extra=3, drop=True, wide=0):
    """Rows in a random order, more than slots name, some slots dropped."""
    g = gen(seed)
    rows = T * k + extra
    inv = torch.randperm(rows, generator=g)[:T * k].to(I32)
    if drop:
        inv[torch.rand(T * k, generator=g) < 0.2] = -1
        inv[torch.rand(T * k, generator=g) < 0.1] = rows
        inv[:k] = -1                      # a token without any slot
    z = normal(g, (rows, d + wide), 1.0, DT[zdt])
    w = torch.softmax(torch.randn((T, k), generator=g), 1)
    add, dy = normal(g, (T, d + wide), 1.0, DT[ydt]), normal(g, (T, d + wide), 1.0, DT[ydt])
    # what must not be read: weights of dropped slots, rows that no slot names
    live = (inv >= 0) & (inv < rows)
    w.view(-1)[~live] = float("nan")
    named = torch.zeros(rows, dtype=torch.bool)
    named[inv[live].long()] = True
    z[~named] = float("nan")
    return rows, inv, z, w, add, dy, live, named


# from 4096 tokens a wave takes a token of up to 2048 or 4096 values
MANY = [(4097, 2, 136), (4100, 3, 2056), (4096, 1, 4104)]
SIZES = [(1, 1, 8), (1, 8, 2048), (3, 2, 136), (32, 4, 2048), (130, 6, 1032), (700, 3, 4096), (5, 9, 5128), (2, 32, 16)]


@pytest.mark.parametrize("T,k,d", SIZES)
@pytest.mark.parametrize("zdt,ydt", [("f16", "f16"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("kind", ["weights", "add", "sum"])
def test_sum(T, k, d, zdt, ydt, kind):
    print(f"[case] combine {T} {k} {d} {zdt} {ydt} {kind}", flush=True)
    wide = 8 if kind == "add" else 0
    rows, inv, z, w, add, _, live, _ = make(T, k, d, zdt, ydt, 1, wide=wide)
    y = torch.full((T, d + wide), -7.0, dtype=DT[ydt], device="cuda")
    tq.combine(z.cuda()[:, :d], inv.cuda(), y[:, :d], w=None if kind == "sum" else w.cuda(),
               add=add.cuda()[:, :d] if kind == "add" else None)
    f = torch.where(live[:, None], z.double()[inv.long().clamp(0, rows - 1)][:, :d], 0.0)
    if kind != "sum":
        f = f * torch.where(live, w.double().view(-1), 0.0)[:, None]
    f = f.view(T, k, d)
    ref, mag = f.sum(1), f.abs().sum(1)
    if kind == "add":
        ref, mag = ref + add.double()[:, :d], mag + add.double()[:, :d].abs()
    check("y", y[:, :d], ref, 1.01 * (k + 1) * U * mag + half_step(ref, DT[ydt]))
    assert (y[:, d:] == -7).all()


@pytest.mark.parametrize("T,k,d", SIZES + MANY)
@pytest.mark.parametrize("zdt,ydt", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("want", ["both", "dz", "dw", "plain"])
def test_gradient(T, k, d, zdt, ydt, want):
    print(f"[case] combine grad {T} {k} {d} {zdt} {ydt} {want}", flush=True)
    wide = 8 if want == "both" else 0
    rows, inv, z, w, _, dy, live, named = make(T, k, d, zdt, ydt, 2, wide=wide)
    dz = torch.full((rows, d + wide), -7.0, dtype=DT[zdt], device="cuda")
    dw = torch.full((T, k), -7.0, device="cuda")
    tq.combine_grad(dy.cuda()[:, :d], inv.cuda().view(T, k), w=None if want == "plain" else w.cuda(),
                    z=z.cuda()[:, :d] if want in ("both", "dw") else None,
                    dz=None if want == "dw" else dz[:, :d], dw=dw if want in ("both", "dw") else None)
    r, t = inv.long().clamp(0, rows - 1), torch.arange(T * k) // k
    dyd = dy.double()[t][:, :d]
    if want in ("both", "dw"):
        p = torch.where(live[:, None], z.double()[r][:, :d] * dyd, 0.0)
        check("dw", dw.view(-1), p.sum(1), (d / 64 + 8 + 8) * U * p.abs().sum(1))
        assert (dw.view(-1).cpu()[~live] == 0).all()
    else:
        assert (dw == -7).all()
    if want != "dw":
        ref = dyd if want == "plain" else w.double().view(-1)[:, None] * dyd
        got = dz[:, :d].cpu()[r[live]]
        check("dz", got, ref[live], 1.01 * U * ref[live].abs() + half_step(ref[live], DT[zdt]))
        dz[torch.nonzero(named)[:, 0].cuda(), :d] = -7.0
    assert (dz == -7).all(), "rows that no slot names, or columns beside them, were written"


def test_more_tokens_than_workgroups():
    """A launch takes 2^24 tokens, one wave each; 2^20 workgroups of four waves take
    slots in turns."""
    T, d = (1 << 24) + 5, 8
    inv = torch.arange(T - 1, -1, -1, dtype=I32, device="cuda")
    z, dy = torch.randn((T, d), device="cuda").half(), torch.randn((T, d), device="cuda").half()
    y, dz, dw = torch.empty_like(z), torch.zeros_like(z), torch.empty((T, 1), device="cuda")
    tq.combine(z, inv, y)
    assert torch.equal(y, z.flip(0))
    tq.combine_grad(dy, inv, z=z, dz=dz, dw=dw)
    assert torch.equal(dz, dy.flip(0))
    p = dy.double() * z.flip(0).double()
    assert ((dw[:, 0].double() - p.sum(1)).abs() <= (8 + 8) * U * p.abs().sum(1)).all()
    del p
    few, k = T // 2048, 2048            # few tokens of many slots: a wave a slot
    tq.combine_grad(dy[:few], inv[:few * k], z=z, dz=dz)
    assert torch.equal(dz.flip(0)[:few * k], dy[:few].repeat_interleave(k, 0))


def test_gradient_against_differences():
    """y is linear in z and in w: y(w + e) - y(w) = e dy^T dw, up to roundings."""
    T, k, d = 6, 3, 64
    rows, inv, z, w, _, dy, live, _ = make(T, k, d, "f32", "f32", 3, drop=False)
    zd, iv, wd, dyd = z.cuda(), inv.cuda(), w.cuda(), dy.cuda()
    dz, dw = torch.zeros_like(zd), torch.empty((T, k), device="cuda")
    tq.combine_grad(dyd, iv, w=wd, z=zd, dz=dz, dw=dw)
    g, loss = gen(4), []
    ez, ew = torch.randn(z.shape, generator=g).cuda(), torch.randn((T, k), generator=g).cuda()
    for s in (1.0, -1.0):
        for a, b in ((s, 0.0), (0.0, s)):
            y = torch.empty((T, d), device="cuda")
            tq.combine(torch.nan_to_num(zd) + a * ez, iv, y, w=wd + b * ew)
            loss.append((y.double() * dyd.double()).sum().item())
    for got, hi, lo in (((dz.double() * ez.double()).sum().item(), loss[0], loss[2]),
                        ((dw.double() * ew.double()).sum().item(), loss[1], loss[3])):
        # (some hundreds of terms of size 1 to 10, each off by a few 2^-24)
        assert abs(got - (hi - lo) / 2) < 2e-3


def test_all_slots_dropped_and_empty_calls():
    T, k, d = 4, 2, 64
    inv = torch.full((T * k,), -1, dtype=I32, device="cuda")
    z, y = torch.full((8, d), float("nan"), device="cuda"), torch.full((T, d), 7.0, device="cuda")
    tq.combine(z, inv, y)
    assert (y == 0).all()
    add = torch.randn((T, d), device="cuda")
    tq.combine(z, inv, y, w=torch.full((T, k), float("nan"), device="cuda"), add=add)
    assert torch.equal(y, add)
    dw, dz = torch.full((T, k), 7.0, device="cuda"), torch.full_like(z, 7.0)
    tq.combine_grad(add, inv, z=z, dz=dz, dw=dw)
    assert (dw == 0).all() and (dz == 7).all()
    # no rows at all
    tq.combine(z[:0], torch.zeros(T * k, dtype=I32, device="cuda"), y)
    assert (y == 0).all()
    none = torch.empty(0, dtype=I32, device="cuda")
    tq.combine(z, none, y[:0])
    tq.combine_grad(y[:0], none, z=z, dz=dz)
    tq.combine(z, none.view(0, k), y[:0])


def test_in_place_and_one_row_twice():
    T, k, d = 40, 3, 264
    rows, inv, z, w, add, dy, live, named = make(T, k, d, "bf16", "bf16", 5)
    zd, iv, wd = z.cuda(), inv.cuda(), w.cuda()
    y, acc = torch.empty((T, d), dtype=torch.bfloat16, device="cuda"), add.cuda().clone()
    tq.combine(zd, iv, y, w=wd, add=add.cuda())
    tq.combine(zd, iv, acc, w=wd, add=acc)
    assert torch.equal(acc, y)
    dz, dw, dw2 = torch.zeros_like(zd), torch.empty((T, k), device="cuda"), torch.empty((T, k), device="cuda")
    tq.combine_grad(dy.cuda(), iv, w=wd, z=zd, dz=dz, dw=dw)
    z2 = zd.clone()
    tq.combine_grad(dy.cuda(), iv, w=wd, z=z2, dz=z2, dw=dw2)
    at = torch.nonzero(named)[:, 0].cuda()
    assert torch.equal(z2[at], dz[at]) and torch.equal(dw, dw2)
    # a row that two slots name counts twice
    two = torch.tensor([5, 5], dtype=I32, device="cuda")
    one = torch.randn((8, d), device="cuda")
    y = torch.empty((1, d), device="cuda")
    tq.combine(one, two, y)
    assert torch.equal(y[0], one[5] + one[5])


def test_graph_and_streams():
    T, k, d = 33, 4, 520
    rows, inv, z, w, add, dy, _, _ = make(T, k, d, "f16", "f16", 6, drop=False)
    zd, iv, wd, ad, dyd = z.cuda(), inv.cuda(), w.cuda(), add.cuda(), dy.cuda()
    y, dz, dw = torch.empty_like(ad), torch.zeros_like(zd), torch.empty((T, k), device="cuda")

    def step(stream=None):
        tq.combine(zd, iv, y, w=wd, add=ad, stream=stream)
        tq.combine_grad(dyd, iv, w=wd, z=zd, dz=dz, dw=dw, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dz, dw)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for how in ("stream", "handle", "graph", "graph", "graph"):
        y.fill_(3)
        dw.fill_(3)
        torch.randn(1000, device="cuda").sum().item()
        torch.cuda.synchronize()
        if how == "graph":
            graph.replay()
        else:
            step(side if how == "stream" else side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(t, v) for t, v in zip((y, dz, dw), want))


def test_the_gradient_of_a_gather():
    """Rows of gradients, one per slot, summed over the slots of a token."""
    T, k, K, d = 50, 3, 8, 128
    g = gen(7)
    ids = torch.stack([torch.randperm(K, generator=g)[:k] for _ in range(T)]).to(I32).cuda()
    off, perm, inv = (torch.empty(n, dtype=I32, device="cuda") for n in (K + 1, T * k, T * k))
    ws = torch.empty(tq.group_slots_workspace(T, k, K), dtype=torch.uint8, device="cuda")
    tq.group_slots(ids, K, off, perm, inv, ws)
    dxr, dx = normal(g, (T * k, d), 1.0, torch.float32).cuda(), torch.empty((T, d), device="cuda")
    tq.combine(dxr, inv, dx)
    rows = dxr.double().cpu()
    tok = perm.long().cpu() // k
    ref = torch.zeros((T, d), dtype=torch.float64).index_add_(0, tok, rows)
    mag = torch.zeros((T, d), dtype=torch.float64).index_add_(0, tok, rows.abs())
    check("dx", dx, ref, 1.01 * (k + 1) * U * mag + half_step(ref, torch.float32))
