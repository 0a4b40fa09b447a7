"""The largest sizes that the operators between and after the products take:
launches in several parts, a layer of 1024 slots and of rows of 65536."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.experts_cases import skewed
from tests.gpu_util import need_gpu
from tests.ops_util import DT, check, gen, half_step, normal
from tests.test_gpu_experts import run
from tests.test_gpu_experts_kernels import whole_reference

pytestmark = pytest.mark.gpu
WIDE = 1 << 24                              # the widest row; 1023 of them are one launch


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def need_memory(gib):
    free = torch.cuda.mem_get_info()[0] / 2 ** 30
    if free < gib + 8:
        pytest.skip(f"{free:.0f} GiB free, {gib} needed")


def test_swiglu_in_several_launches():
    """h in the place of the gates; rows on both sides of the border between two
    launches, beginnings and ends."""
    need_memory(69)
    rows = 1030
    a = torch.zeros((rows, 2 * WIDE), dtype=torch.float16, device="cuda")
    parts = (slice(0, 2), slice(1021, 1025), slice(rows - 2, rows))
    cols = (slice(0, 64), slice(WIDE - 64, WIDE))
    g, want = gen(51), []
    for p in parts:
        for c in cols:
            n = p.stop - p.start
            v = normal(g, (n, 128), 2.0, torch.float16)
            a[p, c] = v[:, :64].cuda()
            a[p, c.start + WIDE:c.stop + WIDE] = v[:, 64:].cuda()
            gate, up = v.double().chunk(2, 1)
            want.append((p, c, gate * torch.sigmoid(gate) * up))
    tq.swiglu(a, a[:, :WIDE])
    for p, c, ref in want:
        check(f"rows {p.start}", a[p, c], ref, 9.5 * 2.0 ** -24 * ref.abs() + half_step(ref, torch.float16))
    assert (a[5:1000:7, 64:WIDE - 64:65521] == 0).all()


def test_sum_over_slots_in_several_launches():
    need_memory(35)
    T = 1030
    z = normal(gen(52), (2, WIDE), 1.0, torch.float16).cuda()
    inv = torch.tensor([[t % 2, -1] if t % 3 else [0, 1] for t in range(T)], dtype=torch.int32, device="cuda")
    y = torch.full((T, WIDE), -7.0, dtype=torch.float16, device="cuda")
    tq.combine(z, inv, y)
    both = (z[0].float() + z[1].float()).half()
    for t in (0, 1, 2, 3, 1021, 1022, 1023, 1024, 1025, T - 2, T - 1):
        assert torch.equal(y[t], z[t % 2] if t % 3 else both), t


# experts, tokens, topk, d, ff, slots of one expert
@pytest.mark.parametrize("E,T,k,d,ff,hot", [(2, 1024, 1, 16, 65536, 700), (3, 64, 16, 65536, 16, 500), (1024, 32, 32, 32, 16, 600),
                                            (1, 1, 1, 65536, 65536, 1), (40, 1, 32, 65536, 16, 5), (1024, 1024, 1, 16, 16, 1)])
@pytest.mark.parametrize("dtype,int8", [("f16", False), ("bf16", True)])
def test_layer(E, T, k, d, ff, hot, dtype, int8):
    if d * ff > 1 << 24 and not int8:
        pytest.skip("the other kind of weights runs this size")
    print(f"[case] layer limits {E} {T} {k} {d} {ff} {hot} {dtype} {int8}", flush=True)
    if d * ff > 1 << 24:                     # (12 GiB of weights: two of the inputs and of ff are not zero)
        need_memory(13)
        w_up, w_down = (torch.zeros(s, dtype=torch.int8, device="cuda") for s in ((1, 2 * ff, d), (1, d, ff)))
        x, w = torch.zeros((1, d), dtype=DT[dtype], device="cuda"), torch.ones((1, 1), device="cuda")
        x[0, 0], x[0, d - 1] = 1.0, 2.0
        w_up[0, :, 0], w_up[0, :, d - 1] = 1, 100       # 201 each, times the scale: 0.785
        w_down[0, :, 0], w_down[0, :, ff - 1] = 3, -100
        y = torch.empty((1, d), device="cuda")
        ws = torch.full((tq.experts_workspace(1, 1, 1, d, ff),), 255, dtype=torch.uint8, device="cuda")
        ids = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        tq.experts_forward(x, ids, w, w_up, w_down, y, ws, s_up=torch.full((1, 2 * ff), 2.0 ** -8, device="cuda"),
                           s_down=torch.ones((1, d), device="cuda"))
        a = torch.tensor(201.0 * 2.0 ** -8, dtype=torch.float64)
        h = (a * a * torch.sigmoid(a)).to(DT[dtype]).double()
        # (h is not next to a border between two values: the f32 result rounds alike)
        assert torch.equal(y.double().cpu(), torch.full((1, d), float(-97 * h), dtype=torch.float64))
        return
    m = skewed(E, T, k, d, ff, hot, DT[dtype], int8, 53, True)
    y = run(m)
    ref, tol = whole_reference(*m, DT[dtype])
    check("y", y, ref, 1.01 * tol + half_step(ref, torch.float32))
