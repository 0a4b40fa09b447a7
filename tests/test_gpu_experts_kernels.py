"""Each kernel of the layer for a few tokens on numbers, in both types and with
both kinds of weights, with 17 and more slots of one expert: several products of
columns after one another in one workgroup.

Bounds as in test_gpu_experts; its d 2^-23 of the magnitudes of a sum is as much
as a step of k that is left out, so the same runs on whole numbers too, whose gate
and up sums a are exact (8-bit weights: one rounding for the scale, 2^-24).  Then
only silu (2^-20), h's rounding and the sum over ff are left."""
import pytest
import torch

from tests.experts_cases import CASES8, CASES16, kernels_of, skewed
from tests.gpu_util import need_gpu
from tests.ops_util import DT, check, half_step
from tests.test_gpu_experts import reference, run

pytestmark = pytest.mark.gpu


def whole_reference(x, ids, w, w_up, w_down, s_up, s_down, dt):
    """y in 64 bits and its bound before the last rounding, of exact gate and up sums."""
    E, d, ff = w_down.shape
    (T, k), xd = ids.shape, x.double()
    y, tol = torch.zeros((T, d), dtype=torch.float64), torch.zeros((T, d), dtype=torch.float64)
    for e in ids.unique().tolist():
        if not 0 <= e < E:
            continue
        t, j = (ids == e).nonzero(as_tuple=True)
        a, v, ea = xd[t] @ w_up[e].double().t(), w_down[e].double(), 0.0
        if s_up is not None:
            a, v, ea = a * s_up[e].double(), v * s_down[e].double()[:, None], 2.0 ** -24
        g, up = a.chunk(2, 1)
        h = g * torch.sigmoid(g) * up
        # (silu's slope is below 1.1)
        eh = 1.1 * ea * (g * up).abs() + ea * h.abs() + 2.0 ** -20 * h.abs()
        eh = eh + half_step(h.abs() + eh, dt)
        h = h.to(dt).double()
        eh = eh + half_step(h, dt)
        c = w[t, j].double()[:, None]
        y.index_add_(0, t, c * (h @ v.t()))
        tol.index_add_(0, t, c * ((ff + k + 4) * 2.0 ** -23 * (h.abs() @ v.abs().t()) + eh @ v.abs().t()))
    return y, tol


@pytest.mark.parametrize("case", [c + (int8,) for int8, cs in ((False, CASES16), (True, CASES8)) for c in cs],
                         ids=lambda c: f"{'int8' if c[-1] else '16'}-{c[0]}-{'x'.join(map(str, c[1] + c[2]))}-{c[8]}of{c[3]}")
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("whole", [False, True])
def test_each_kernel(case, dtype, whole):
    need_gpu()
    columns, up, down, E, T, k, d, ff, hot, int8 = case
    assert kernels_of(T, k, E, d, ff, int8) == (columns, up, down)
    print(f"[case] layer kernels {case} {dtype} {whole}", flush=True)
    m = skewed(E, T, k, d, ff, hot, DT[dtype], int8, 41, whole)
    assert int(torch.bincount(m[1][m[1] >= 0]).max()) >= hot
    y = run(m)
    ref, tol = (whole_reference if whole else reference)(*m, DT[dtype])
    check("y", y, ref, 1.01 * tol + half_step(ref, torch.float32))
    assert torch.equal(run(m, "bf16"), y.to(torch.bfloat16))
