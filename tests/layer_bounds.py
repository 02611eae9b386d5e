"""Error bounds of the operators around the SSD, from the arithmetic they do.

U is fp32's largest relative error of one operation, 2^-24; RND the rounding of
an output to its dtype, half a unit: 2^-8 for bf16, and for fp32 the one U that
the last operation already has.  A bound counts the operations between input
and output, each with one U of its operands' size (sums: of the sum of absolute
values), and what the hardware's functions add: exp within 2 units in the last
place (4 U) plus the rounding of its argument z log2(e) (2 |z| U), reciprocal
and reciprocal square root 1 unit (2 U).
"""
import numpy as np
import torch

U = 2.0 ** -24
TINY = 2.0 ** -120          # results below fp32's normal range may flush to zero
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RND = {"bf16": 2.0 ** -8, "f32": U}


def check(got, ref, tol, what):
    """|got - ref| <= tol in every element (ref NaN: not looked at)."""
    g = got.detach().cpu().double().numpy()
    keep = ~np.isnan(ref)
    err = np.abs(g - ref)
    tol = np.broadcast_to(tol, ref.shape)
    bad = keep & ~(err <= tol)
    worst = float(np.max((err / np.maximum(tol, 1e-300))[keep])) if keep.any() else 0.0
    print(f"  {what}: worst error / bound = {worst:.3f}", flush=True)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first at "
                           f"{tuple(int(v) for v in np.argwhere(bad)[0])}: got {g[bad][0]!r}, "
                           f"expected {ref[bad][0]!r} within {tol[bad][0]:.3e}")


def sigmoid_err(z):
    """Relative error of sigmoid(z): that of e^-z weighs by its share of 1 + e^-z."""
    share = 1.0 / (1.0 + np.exp(np.clip(z, -700, 700)))
    return (share * (4 + 2 * np.abs(z)) + 4) * U
