"""The operators around a layer and the sizes of their workspaces are offered by
the package itself."""
import pytest

import bit_rank_post_amd as tq
from bit_rank_post_amd import ops


@pytest.mark.parametrize("name", ["group_gemm", "group_gemm_dx", "group_gemm_dw", "fp8_gemm", "fp8_quant_rows",
                                  "fp8_quant_blocks", "norm_residual", "norm_residual_grad", "norm_grad_workspace",
                                  "group_slots", "group_slots_workspace"])
def test_offered(name):
    assert getattr(tq, name) is getattr(ops, name)
