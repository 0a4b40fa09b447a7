"""Inputs of the norm gradients as the forward leaves them."""
import torch

import bit_rank_post_amd as tq
from tests.test_gpu_norm import inputs


def prepared(T, d, types, gate, seed):
    """Inputs on the GPU and what the forward leaves for the gradients."""
    s = {k: (v.cuda() if v is not None else None) for k, v in inputs(T, d, *types, gate, seed=seed).items()}
    y, n = torch.empty_like(s["x"]), torch.empty_like(s["b"])
    rp, rn = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    tq.norm_residual(s["x"], y=y, n=n, b=s["b"], w_post=s["w_post"], w_next=s["w_next"], gate=s["gate"],
                     alpha=0.75, rstd_post=rp, rstd_next=rn)
    kw = dict(b=s["b"], w_post=s["w_post"], w_next=s["w_next"], gate=s["gate"], alpha=0.75, rstd_post=rp,
              rstd_next=rn)
    out = dict(dx=torch.empty_like(s["x"]), db=torch.empty_like(s["b"]), dw_post=torch.empty(d, device="cuda"),
               dw_next=torch.empty(d, device="cuda"))
    if gate != "none":
        out["dgate"] = torch.empty_like(s["gate"])
    return s, y, kw, out
