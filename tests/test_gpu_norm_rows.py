"""Norm gradients where a wave or workgroup takes many rows."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.norm_cases import prepared
from tests.ops_util import check, half_step
from tests.test_gpu_norm import U, grad_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


# three rows and more for each wave (d <= 512: 4096 waves) or workgroup (512 or
# 256 of them and up), with a last round that is not full
@pytest.mark.parametrize("T,d", [(13003, 64), (8200, 512), (9001, 512), (3500, 2048), (700, 8192), (800, 8200),
                                 (600, 16384)])
@pytest.mark.parametrize("types,gate", [(("bf16", "bf16", "bf16"), "token"), (("f32", "f16", "f32"), "full"),
                                        (("f32", "f32", "f32"), "none")])
def test_many_rows(T, d, types, gate):
    print(f"[case] norm gradient {T} {d} {types} {gate}", flush=True)
    s, y, kw, out = prepared(T, d, types, gate, 9)
    tq.norm_residual_grad(y, dy=s["dy"], dn=s["dn"], **kw, **out)
    rp, rn = (kw[k].double()[:, None] for k in ("rstd_post", "rstd_next"))
    ref = grad_ref(s, y.double(), rp, rn, 0.75)
    # A sum's error is its depth (the additions that one term goes through) times
    # U: over a row 16 terms a thread, 6 steps of a wave and 16 waves; over the
    # rows at most 4 a wave or workgroup, 3 waves, 8 + 2 parts a run and 32
    # runs.  Two of the former, one of the latter, 12 roundings of single values:
    # less than one row's share of a sum over rows, so that none may be missed.
    depth = 2 * (16 + 6 + 16) + (4 + 3 + 8 + 2 + 32) + 12
    assert depth * U < 0.25 / T
    for name, t in out.items():
        r, mag = ref[name]
        check(name, t, r.cpu(), (depth * U * mag + half_step(r, t.dtype)).cpu())
    # the same bits in place, where a row is written while later ones are read ahead
    dx, db = s["dy"].clone(), s["dn"].clone()
    again = {k: torch.empty_like(v) for k, v in out.items() if k not in ("dx", "db")}
    tq.norm_residual_grad(y, dy=dx, dn=db, dx=dx, db=db, **kw, **again)
    for name, t in dict(again, dx=dx, db=db).items():
        assert torch.equal(t, out[name]), name
