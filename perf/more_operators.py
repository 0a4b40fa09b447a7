"""More operators of a layer of experts, as cases that can be timed: products in
8-bit integers with a scale for each token and channel, SwiGLU between the two
products and its gradient, the sum over a token's slots and its gradient, and a
whole layer for a few tokens.

``run`` computes a case in plain torch (``own`` false) or with this package's
kernels (``own`` true); ``exact`` computes it in 64 bits.

Formulas.  Slot t * topk + j is choice j of token t; off[g] .. off[g+1]-1 are the
rows of expert g, s(r) the token of row r, inv the row of each slot.
  int8          c = max|x| of a row / 127, q = rint(x / c);
                y[r][o] = c_x[s(r)] c_w[g,o] (q_x . q_w)
  int8_down     h = silu(a_gate) a_up quantised the same way, then its int8 product
  swiglu        h = silu(a_gate) a_up, a_gate the first half of a row of a
  swiglu_grad   da from dh, and h again
  combine       y[t] = add[t] + sum_j w[t][j] z[inv[t topk + j]]
  combine_grad  dz[inv[t topk + j]] = w[t][j] dy[t],  dw[t][j] = dy[t] . z[inv[t topk + j]]
  layer         h[t][j] = silu(W_gate x_t) W_up x_t, rounded to x's type, of expert ids[t][j];
                y[t] = sum_j w[t][j] W_down h[t][j];  8-bit weights: c_w[e,o] q_w
"""
import math

import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token through one wide 8-bit matrix, quantised on the way in
        dict(name="int8 one token", op="int8", groups=1, tokens=1, topk=1, d_in=4096, d_out=14336,
             dtype="bf16", routing="uniform", gather=False),
        # prefill of 4160 tokens over 64 small experts with skewed routing
        dict(name="int8 experts ragged", op="int8", groups=64, tokens=4160, topk=6, d_in=2048,
             d_out=1408, dtype="f16", routing="zipf", gather=True),
        # a large dense product in 8 bits
        dict(name="int8 dense large", op="int8", groups=1, tokens=16384, topk=1, d_in=4096,
             d_out=14336, dtype="bf16", routing="uniform", gather=False),
        # the second half of such a layer of experts: activation, quantisation, down product
        dict(name="int8 down ragged", op="int8_down", groups=64, tokens=4160, topk=6, ff=1408, d=2048,
             dtype="f16", routing="zipf"),
        # the activation alone, for a prefill of 16384 tokens through two large experts each
        dict(name="swiglu large", op="swiglu", rows=32768, ff=14336, dtype="bf16", out="bf16"),
        # the activation at decode: 32 tokens through four small experts each
        dict(name="swiglu decode", op="swiglu", rows=128, ff=1408, dtype="f16", out="f16"),
        # its gradient in a training step of the small experts (h is made again for
        # the gradient of the down weights)
        dict(name="swiglu grad", op="swiglu_grad", rows=24960, ff=1408, dtype="bf16", out="f32"),
        # the sum over the slots at decode, where only latency counts
        dict(name="combine decode", op="combine", tokens=32, topk=4, d=2048, dtype="f16", out="f16",
             weights=True, add=False),
        # for a prefill of 16384 tokens, with a shared expert's output added
        dict(name="combine prefill", op="combine", tokens=16384, topk=2, d=4096, dtype="bf16",
             out="bf16", weights=True, add=True),
        # its gradient in a training step of the small experts
        dict(name="combine grad", op="combine_grad", tokens=4160, topk=6, d=2048, dtype="bf16",
             out="bf16"),
        # decode of 32 tokens, four of 60 small experts each
        dict(name="layer 32 tokens", op="layer", experts=60, tokens=32, topk=4, d=2048, ff=1408,
             dtype="f16", weight="16"),
        # decode of one token through two of eight large experts with 8-bit weights
        dict(name="layer int8 one token", op="layer", experts=8, tokens=1, topk=2, d=4096, ff=14336,
             dtype="bf16", weight="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int8", "int8", "int8_down", "swiglu", "swiglu_grad", "combine", "combine_grad", "layer",
                     "layer", "layer"])
    dtype = rng.choice(["f16", "bf16"])
    while True:
        if op == "int8":
            groups = _log(rng, 1, 96)
            case = dict(op=op, groups=groups, tokens=_log(rng, 1, 16384), topk=rng.randint(1, min(groups, 8)),
                        d_in=16 * _log(rng, 8, 512), d_out=8 * _log(rng, 16, 1792), dtype=dtype,
                        routing=rng.choice(["uniform", "zipf", "hot"]), gather=rng.random() < 0.5)
            rows, i, o = case["tokens"] * case["topk"], case["d_in"], case["d_out"]
            if groups * i * o <= 6e8 and rows * max(i, o) <= 4e8 and rows * i * o <= 9e11:
                return case
        elif op == "int8_down":
            groups = _log(rng, 1, 96)
            case = dict(op=op, groups=groups, tokens=_log(rng, 1, 16384), topk=rng.randint(1, min(groups, 8)),
                        ff=16 * _log(rng, 8, 896), d=8 * _log(rng, 16, 1024), dtype=dtype,
                        routing=rng.choice(["uniform", "zipf", "hot"]))
            rows, i, o = case["tokens"] * case["topk"], case["ff"], case["d"]
            if groups * i * o <= 6e8 and rows * max(i, o) <= 2e8 and rows * i * o <= 9e11:
                return case
        elif op in ("swiglu", "swiglu_grad"):
            case = dict(op=op, rows=_log(rng, 1, 65536), ff=8 * _log(rng, 8, 1792), dtype=dtype,
                        out=rng.choice([dtype, dtype, "f32"]))
            if case["rows"] * case["ff"] <= 2e8:
                return case
        elif op == "combine":
            case = dict(op=op, tokens=_log(rng, 1, 16384), topk=rng.randint(1, 8), d=8 * _log(rng, 16, 1024),
                        dtype=rng.choice([dtype, "f32"]), out=dtype, weights=rng.random() < 0.7,
                        add=rng.random() < 0.5)
            if case["tokens"] * case["topk"] * case["d"] <= 2e8:
                return case
        elif op == "combine_grad":
            case = dict(op=op, tokens=_log(rng, 1, 16384), topk=rng.randint(1, 8), d=8 * _log(rng, 16, 1024),
                        dtype=dtype, out=rng.choice([dtype, "f32"]))
            if case["tokens"] * case["topk"] * case["d"] <= 1.5e8:
                return case
        else:
            experts = _log(rng, 2, 128)
            case = dict(op=op, experts=experts, tokens=_log(rng, 1, 64), topk=rng.randint(1, min(experts, 8)),
                        d=16 * _log(rng, 16, 320), ff=16 * _log(rng, 16, 896), dtype=dtype,
                        weight=rng.choice(["16", "16", "int8"]))
            if experts * case["d"] * case["ff"] <= 6e8:
                return case


# ---- inputs ------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, scale, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(0.0, scale, generator=g)


def _popularity(routing, G):
    """How often each expert is chosen, up to a factor."""
    if routing == "zipf":       # falls with the rank
        return [1.0 / e ** 1.1 for e in range(1, G + 1)]
    if routing == "hot":        # one expert in seven of ten choices
        return [0.7] + [0.3 / max(G - 1, 1)] * (G - 1)
    return [1.0] * G


def _ids(g, routing, G, T, k):
    """k different experts for each token, int32 [T][k]."""
    p = torch.tensor(_popularity(routing, G), device="cuda")[torch.randperm(G, device="cuda", generator=g)]
    u = torch.rand((T, G), device="cuda", generator=g).clamp_(1e-7, 1 - 1e-7)
    return (p.log() - (-u.log()).log()).topk(k, dim=1).indices.to(torch.int32)


def _group(ids, G):
    """Expert offsets, the slots in expert order, and each slot's row."""
    flat = ids.reshape(-1).long()
    perm = torch.argsort(flat, stable=True)
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(flat, minlength=G).cumsum(0)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(len(perm), device="cuda")
    return off, perm.to(torch.int32), inv.to(torch.int32)


def _weights8(g, shape, act):
    """Weights in 8-bit integers with a scale for each output channel."""
    q = torch.empty(shape, dtype=torch.int8, device="cuda")
    scale = torch.empty(shape[:-1], device="cuda")
    for e in range(shape[0]):
        w = _normal(g, shape[1:], shape[-1] ** -0.5, act).float()
        scale[e] = w.abs().amax(dim=1) / 127.0
        q[e] = torch.round(w / scale[e][:, None]).to(torch.int8)
    return q, scale


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    act = DTYPE[case["dtype"]]
    s = dict(case=case)
    if op in ("swiglu", "swiglu_grad"):
        rows, ff = case["rows"], case["ff"]
        s["a"] = _normal(g, (rows, 2 * ff), 1.2, act)
        s["h"] = torch.empty((rows, ff), dtype=act if op == "swiglu_grad" else DTYPE[case["out"]], device="cuda")
        if op == "swiglu_grad":
            s["dh"] = _normal(g, (rows, ff), 1.0, DTYPE[case["out"]])
            s["da"] = torch.empty_like(s["a"])
        return s
    if op in ("combine", "combine_grad"):
        T, k, d = case["tokens"], case["topk"], case["d"]
        out = DTYPE[case["out"]]
        s["z"] = _normal(g, (T * k, d), 1.0, act)
        s["inv"] = _group(_ids(g, "uniform", 64, T, k), 64)[2]
        s["w"] = None
        if case.get("weights", True):
            s["w"] = torch.softmax(_normal(g, (T, k), 1.0, torch.float32), dim=1)
        if op == "combine":
            s["add"] = _normal(g, (T, d), 1.0, out) if case["add"] else None
            s["y"] = torch.empty((T, d), dtype=out, device="cuda")
        else:
            s["dy"] = _normal(g, (T, d), 1.0, out)
            s["dz"], s["dw"] = torch.empty_like(s["z"]), torch.empty((T, k), device="cuda")
        return s
    if op == "layer":
        E, T, k, d, ff = (case[n] for n in ("experts", "tokens", "topk", "d", "ff"))
        s["x"] = _normal(g, (T, d), 1.0, act)
        s["ids"] = _ids(g, "uniform", E, T, k)
        s["w"] = torch.softmax(_normal(g, (T, k), 1.0, torch.float32), dim=1)
        s["s_up"] = s["s_down"] = None
        if case["weight"] == "int8":
            s["w_up"], s["s_up"] = _weights8(g, (E, 2 * ff, d), act)
            s["w_down"], s["s_down"] = _weights8(g, (E, d, ff), act)
        else:
            s["w_up"] = _normal(g, (E, 2 * ff, d), d ** -0.5, act)
            s["w_down"] = _normal(g, (E, d, ff), ff ** -0.5, act)
        s["y"] = torch.empty_like(s["x"])
        s["ws"] = None          # made by the first pass of the package's form, and kept
        return s
    G, T, k = case["groups"], case["tokens"], case["topk"]
    rows = T * k
    s["off"], perm, _ = _group(_ids(g, case["routing"], G, T, k), G)
    s["bounds"] = s["off"].tolist()
    if op == "int8":
        di, do = case["d_in"], case["d_out"]
        s["src"], s["div"] = (perm, k) if case["gather"] else (None, 1)
        s["x"] = _normal(g, (T if case["gather"] else rows, di), 1.0, act)
    else:
        di, do = case["ff"], case["d"]
        s["a"] = _normal(g, (rows, 2 * di), 1.2, act)
    n = len(s["x"] if op == "int8" else s["a"])
    s["w"], s["w_scale"] = _weights8(g, (G, do, di), act)
    s["y"] = torch.empty((rows, do), dtype=act, device="cuda")
    s["q"], s["q_scale"] = torch.empty((n, di), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------


def _quant(x):
    """Rows in 32 bits to the values of their 8-bit codes, and the scales."""
    # the division is that of the definition, also where it ends next to a
    # border between two codes (a product with 1/127 moves some across)
    scale = (x.abs().amax(dim=1).double() / 127.0).float()
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return torch.round(x / scale[:, None]), scale


def _product8(s, q, scale):
    if s.get("src") is not None:
        row = s["src"].long() // s["div"]
        q, scale = q[row], scale[row]
    y = torch.empty((len(q), s["w"].shape[1]), device="cuda")
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if hi > lo:
            y[lo:hi] = q[lo:hi] @ s["w"][e].float().t() * s["w_scale"][e]
    return (y * scale[:, None]).to(s["y"].dtype)


def _silu_mul(a):
    gate, up = a.float().chunk(2, dim=1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _swiglu_grad(s):
    gate, up = s["a"].float().chunk(2, dim=1)
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    da = torch.cat([dh * up * (sig * (1.0 + gate * (1.0 - sig))), dh * (gate * sig)], dim=1)
    return [da.to(s["a"].dtype), (gate * sig * up).to(s["h"].dtype)]


def _combine(s):
    T, k, d = (s["case"][n] for n in ("tokens", "topk", "d"))
    z = s["z"][s["inv"].long()].view(T, k, d).float()
    y = z.sum(dim=1) if s["w"] is None else (z * s["w"][:, :, None]).sum(dim=1)
    return (y if s["add"] is None else y + s["add"].float()).to(s["y"].dtype)


def _combine_grad(s):
    T, k, d = (s["case"][n] for n in ("tokens", "topk", "d"))
    inv, dy = s["inv"].long(), s["dy"].float()
    dw = (s["z"][inv].view(T, k, d).float() * dy[:, None, :]).sum(dim=2)
    dz = torch.empty_like(s["z"])
    dz[inv] = (s["w"][:, :, None] * dy[:, None, :]).view(T * k, d).to(dz.dtype)
    return [dz, dw]


def _layer(s):
    E, T, k, d, ff = (s["case"][n] for n in ("experts", "tokens", "topk", "d", "ff"))
    x, act = s["x"].float(), s["x"].dtype

    def weights(w, scale, pick):
        w = w[pick].float()
        return w if scale is None else w * scale[pick][:, :, None]

    if T * k <= E:      # the experts of each slot
        pick = s["ids"].reshape(-1).long()
        cols = x.repeat_interleave(k, dim=0)[:, :, None]
    else:               # all experts on all tokens
        pick = torch.arange(E, device="cuda")
        cols = x.t().contiguous()[None].expand(E, d, T)
    a = torch.bmm(weights(s["w_up"], s["s_up"], pick), cols)
    h = a[:, :ff] / (1.0 + torch.exp(-a[:, :ff])) * a[:, ff:]
    o = torch.bmm(weights(s["w_down"], s["s_down"], pick), h.to(act).float())
    if T * k <= E:
        return (o.view(T, k, d) * s["w"][:, :, None]).sum(dim=1).to(act)
    dense = torch.zeros((T, E), device="cuda").scatter_add_(1, s["ids"].long(), s["w"])
    return (o * dense.t()[:, None, :]).sum(dim=0).t().contiguous().to(act)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "int8":
            return _product8(s, *_quant(s["x"].float()))
        if op == "int8_down":
            return _product8(s, *_quant(_silu_mul(s["a"])))
        if op == "swiglu":
            return _silu_mul(s["a"]).to(s["h"].dtype)
        return {"swiglu_grad": _swiglu_grad, "combine": _combine, "combine_grad": _combine_grad,
                "layer": _layer}[op](s)
    import bit_rank_post_amd as tq
    if op == "int8":
        tq.int8_quant_rows(s["x"], s["q"], s["q_scale"])
        tq.int8_gemm(s["q"], s["q_scale"], s["w"], s["w_scale"], s["y"], off=s["off"], src=s["src"],
                     src_div=s["div"])
        return s["y"]
    if op == "int8_down":
        tq.swiglu_int8(s["a"], s["q"], s["q_scale"], off=s["off"])
        tq.int8_gemm(s["q"], s["q_scale"], s["w"], s["w_scale"], s["y"], off=s["off"])
        return s["y"]
    if op == "swiglu":
        tq.swiglu(s["a"], s["h"])
        return s["h"]
    if op == "swiglu_grad":
        tq.swiglu_grad(s["a"], s["dh"], s["da"], h=s["h"])
        return [s["da"], s["h"]]
    if op == "combine":
        tq.combine(s["z"], s["inv"], s["y"], w=s["w"], add=s["add"])
        return s["y"]
    if op == "combine_grad":
        tq.combine_grad(s["dy"], s["inv"], w=s["w"], z=s["z"], dz=s["dz"], dw=s["dw"])
        return [s["dz"], s["dw"]]
    if s["ws"] is None:
        c = s["case"]
        s["ws"] = torch.empty(tq.experts_workspace(c["tokens"], c["topk"], c["experts"], c["d"], c["ff"]),
                              dtype=torch.uint8, device="cuda")
    tq.experts_forward(s["x"], s["ids"], s["w"], s["w_up"], s["w_down"], s["y"], s["ws"], s_up=s["s_up"],
                       s_down=s["s_down"])
    return s["y"]


def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}
    a, op = size[case["dtype"]], case["op"]
    if op in ("swiglu", "swiglu_grad"):
        n, o = case["rows"] * case["ff"], size[case["out"]]
        if op == "swiglu":
            return {"bytes": n * (2 * a + o), "flops": 6 * n}
        return {"bytes": n * (2 * a + o + 2 * a + a), "flops": 14 * n}
    if op in ("combine", "combine_grad"):
        T, S, d, o = case["tokens"], case["tokens"] * case["topk"], case["d"], size[case["out"]]
        if op == "combine":
            return {"bytes": S * d * a + T * d * o * (2 if case["add"] else 1) + 4 * S * (2 if case["weights"] else 1),
                    "flops": 2 * S * d}
        return {"bytes": 2 * S * d * a + T * d * o + 12 * S, "flops": 3 * S * d}
    if op == "layer":
        E, T, k, d, ff = (case[n] for n in ("experts", "tokens", "topk", "d", "ff"))
        # the experts that are expected to be chosen at all
        hit = max(k, round(E * (1 - (1 - k / E) ** T)))
        w = hit * 3 * d * ff * (1 if case["weight"] == "int8" else a)
        return {"bytes": w + (hit * (2 * ff + d) * 4 if case["weight"] == "int8" else 0) + 2 * T * d * a + 8 * T * k,
                "flops": 6 * T * k * d * ff}
    G, T, k = case["groups"], case["tokens"], case["topk"]
    rows = T * k
    p = _popularity(case["routing"], G)
    active = min(G, rows, max(k, round(sum(1 - (1 - v / sum(p)) ** rows for v in p))))
    if op == "int8":
        di, do = case["d_in"], case["d_out"]
        xb = (T if case["gather"] else rows) * di * a + (4 * rows if case["gather"] else 0)
    else:
        di, do = case["ff"], case["d"]
        xb = rows * 2 * di * a
    return {"bytes": xb + active * do * (di + 4) + rows * do * a, "flops": 2 * rows * di * do}


# ---- the definition in 64 bits -------------------------------------------------


def _codes(v):
    """Rows in 64 bits to the values that their 8-bit codes stand for."""
    unit = (v.abs().amax(1, keepdim=True) / 127).float().to(v.dtype)
    unit[unit == 0] = 1.0
    return torch.round((v / unit).float().to(v.dtype)) * unit


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    D = torch.float64
    if op == "swiglu":
        ff = case["ff"]
        parts = [p[:, :ff] * torch.sigmoid(p[:, :ff]) * p[:, ff:] for p in map(lambda t: t.to(D), s["a"].split(4096))]
        return torch.cat(parts)
    if op == "swiglu_grad":
        a = s["a"].to(D).view(case["rows"], 2, case["ff"]).requires_grad_()
        h = torch.nn.functional.silu(a[:, 0]) * a[:, 1]
        da, = torch.autograd.grad(h, a, s["dh"].to(D))
        return [da.view(case["rows"], -1), h.detach()]
    if op == "combine":
        y = torch.zeros(s["y"].shape, dtype=D, device="cuda") if s["add"] is None else s["add"].to(D)
        for j in range(case["topk"]):
            row = s["z"][s["inv"][j::case["topk"]].long()].to(D)
            y += row if s["w"] is None else row * s["w"][:, j:j + 1].to(D)
        return y
    if op == "combine_grad":
        dz = torch.zeros(s["z"].shape, dtype=D, device="cuda")
        dw = torch.zeros(s["dw"].shape, dtype=D, device="cuda")
        dy = s["dy"].to(D)
        for j in range(case["topk"]):
            at = s["inv"][j::case["topk"]].long()
            dz.index_copy_(0, at, dy * s["w"][:, j:j + 1].to(D))
            dw[:, j] = torch.linalg.vecdot(dy, s["z"].index_select(0, at).to(D))
        return [dz, dw]
    if op == "layer":
        y = torch.zeros(s["y"].shape, dtype=D, device="cuda")
        for e in s["ids"].unique().tolist():
            t, j = (s["ids"] == e).nonzero(as_tuple=True)
            w1, w2 = s["w_up"][e].to(D), s["w_down"][e].to(D)
            if s["s_up"] is not None:
                w1, w2 = s["s_up"][e].to(D).unsqueeze(1) * w1, s["s_down"][e].to(D).unsqueeze(1) * w2
            v = s["x"][t].to(D).matmul(w1.t())
            h = torch.nn.functional.silu(v[:, :case["ff"]]) * v[:, case["ff"]:]
            y.index_add_(0, t, h.to(s["x"].dtype).to(D).matmul(w2.t()) * s["w"][t, j].to(D).unsqueeze(1))
        return y
    if op == "int8":
        x, src = _codes(s["x"].to(D)), s["src"]
        if src is not None:
            x = x.index_select(0, torch.div(src, s["div"], rounding_mode="floor"))
    else:
        v = s["a"].to(D)
        x = _codes(torch.nn.functional.silu(v[:, :case["ff"]]) * v[:, case["ff"]:])
    y = torch.empty(s["y"].shape, dtype=D, device="cuda")
    for e, w in enumerate(s["w"]):
        lo, hi = s["bounds"][e:e + 2]
        y[lo:hi] = x[lo:hi].matmul((w.to(D) * s["w_scale"][e].to(D).unsqueeze(1)).t())
    return y
