"""Helpers for the tests of the operators around a layer: ragged offsets, and
error bounds that follow from the arithmetic.

Bounds.  A product of two 16-bit values (11 or 8 significand bits) is exact in
f32; a sum of K of them in f32, in any order and with truncation at each step,
is off by at most K 2^-23 sum|a b|.  The result is then rounded once: half a
step, eps/2 of its value, or half the smallest subnormal."""
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def half_step(value, dtype):
    """What one rounding of `value` to dtype may add."""
    f = torch.finfo(dtype)
    # value is the exact result: what is rounded differs from it by less than
    # the accumulation bound, whose own rounding is second order (the 1.01)
    return 1.01 * value.abs() * f.eps / 2 + f.smallest_normal * f.eps / 2


def check(name, got, ref, tol):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= tol)           # also where something is not a number
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    print(f"  {name}: max error {float(err.max()) if err.numel() else 0:.3g}, worst error/bound {worst:.3f}",
          flush=True)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} values off, worst {worst:.3f} of the bound"


def offsets(counts, lead=0):
    off = [lead]
    for c in counts:
        off.append(off[-1] + c)
    return off


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, shape, scale, dtype):
    return (torch.randn(shape, generator=g) * scale).to(dtype)
