"""The sum over a token's experts is made by the workgroup that comes last, from
what the others left in the workspace.  Before each call the workspace holds
NaN or the sums of other inputs of the same sizes, so that a sum that is read
before it has arrived shows in the result; the results are compared with the
formula, too."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import check, half_step
from tests.test_gpu_experts import make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# many workgroups that end together; several products of columns; few workgroups
SIZES = [(60, 24, 4, 512, 264, "bf16", False), (8, 40, 2, 1024, 144, "f16", True), (4, 64, 2, 528, 96, "f16", False),
         (64, 3, 8, 2048, 48, "bf16", True)]


def prepared(E, T, k, d, ff, dtype, int8):
    a, b = make(E, T, k, d, ff, dtype, int8, 31, repeat=True), make(E, T, k, d, ff, dtype, int8, 32, repeat=True)
    out = []
    for m in (a, b):
        ref, tol = reference(*m, m[0].dtype)
        c = [None if t is None else t.cuda() for t in m]
        out.append((c, ref, 1.01 * tol + half_step(ref, torch.float32)))
    return out, tq.experts_workspace(T, k, E, d, ff)


def call(c, y, ws, stream=None):
    tq.experts_forward(*c[:5], y, ws, s_up=c[5], s_down=c[6], stream=stream)


@pytest.mark.parametrize("E,T,k,d,ff,dtype,int8", SIZES)
def test_no_sum_is_read_before_it_arrives(E, T, k, d, ff, dtype, int8):
    print(f"[case] layer workspace {E} {T} {k} {d} {ff} {dtype} {int8}", flush=True)
    inputs, n = prepared(E, T, k, d, ff, dtype, int8)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")       # (all ones: NaN in f32 and in 16 bits)
    want = []
    for c, ref, tol in inputs:
        y = torch.full((T, d), float("nan"), device="cuda")
        ws.fill_(255)
        call(c, y, ws)
        check("y", y, ref, tol)
        want.append(y.clone())
    assert not torch.equal(*want)
    for i in range(60):
        y.fill_(float("nan"))
        if i % 3 == 0:
            ws.fill_(255)
        call(inputs[i % 2][0], y, ws)           # else: the other inputs' sums lie there
        assert torch.equal(y, want[i % 2]), i


def test_two_streams_each_with_its_workspace():
    E, T, k, d, ff, dtype, int8 = SIZES[0]
    inputs, n = prepared(E, T, k, d, ff, dtype, int8)
    side = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = [[torch.full((T, d), float("nan"), device="cuda") for _ in range(12)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(12):
        for s in range(2):
            with torch.cuda.stream(side[s]):
                if i % 3 == 0:
                    ws[s].fill_(255)
                call(inputs[(i + s) % 2][0], ys[s][i], ws[s])
    torch.cuda.synchronize()
    for s in range(2):
        for i, y in enumerate(ys[s]):
            _, ref, tol = inputs[(i + s) % 2]
            check(f"stream {s} call {i}", y, ref, tol)
            assert torch.equal(y, ys[s][i % 2])
