"""Inputs and tolerances of the gated delta rule's tests.

Tolerances, from what the chunked form rounds to fewer bits:
  fp32 inputs: nothing.  Outputs and gradients as the SSD's, relative L2 1e-5 and 1e-4.
  bf16 inputs: every operand on the way to a state is a pair of bf16, off by at most 2^-17 of
    the value, and a product of two pairs, without the two low parts', by 2^-16 more.  A chunk
    adds to a state what passes six units of 2^-17 (the state, what it leaves of v, the matrix
    1 / (1 + L) and its product with that, the rows w decayed), so 2^-14; the gradient of the
    starting state as much by itself and on the forward's side, 2^-13, and the gradients of
    fp32 gates, sums over both of them, 2^-13.
    What is rounded to bf16 once on the way (the output and the gradients of q, k, v, and of
    bf16 gates over many tokens) is held to the SSD's bf16 tolerance.
"""
import numpy as np
import torch

from oracle import delta
from oracle.recurrence import seq_ranges
from tests.helpers import assert_close, f64
from tests.layer_bounds import TINY

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL_STATE = {"f32": 1e-5, "bf16": 2.0 ** -14}
TOL_GATE = {"f32": 1e-4, "bf16": 2.0 ** -13}


def unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


def draw(b=1, T=100, H=4, G=2, P=32, N=64, dtype="bf16", gate="f32", nseq=None, init=True, seed=0,
         decay=0.1):
    """On the CPU.  Keys and queries of unit length, beta in (0, 1), g <= 0."""
    r = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    t, gt = DT[dtype], DT[gate]
    n = b if nseq is None else nseq
    return dict(q=unit(rn(b, T, G, N)).to(t), k=unit(rn(b, T, G, N)).to(t), v=rn(b, T, H, P).to(t),
                g=(-decay * rn(b, T, H).abs()).to(gt), beta=torch.rand((b, T, H), generator=r).to(gt),
                initial_states=0.3 * rn(n, H, P, N) if init else None)


def draw_grads(x, seed=1):
    r = torch.Generator().manual_seed(seed)
    b, T, H, P = x["v"].shape
    n = x["initial_states"].shape[0] if x["initial_states"] is not None else None
    dout = torch.randn(x["v"].shape, generator=r).to(x["v"].dtype)
    dfin = None if n is None else torch.randn((n, H, P, x["q"].shape[-1]), generator=r)
    return dout, dfin


def within(got, ref, tol, what):
    """Relative L2 to tol.  What is below fp32's range (its smallest normal number is 2^-126; a
    decay of e^-200 is 2^-288) is zero in the result, whatever its relative size: TINY, 2^-120
    for sums of up to 64 such terms, each element."""
    e, size = np.linalg.norm((f64(got) - f64(ref)).ravel()), np.linalg.norm(f64(ref).ravel())
    print(f"  {what}: error {e:.3e} of {size:.3e}, relative {e / max(size, 1e-300):.3e}", flush=True)
    assert e <= tol * size + TINY * f64(ref).size ** 0.5, what


def dev(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def oracle_fwd(x, scale, cu=None):
    out, fin, _, _ = delta.delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["initial_states"], cu)
    return out, fin


def oracle_bwd(x, dout, dfin, scale, cu=None):
    return delta.delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], dout, scale, x["initial_states"], cu, dfin)


def inside(x, cu):
    """Which tokens belong to a sequence."""
    b, T = x["v"].shape[:2]
    m = torch.zeros(b * T, dtype=torch.bool)
    for at, n in zip(*seq_ranges(b, T, cu)):
        m[at:at + n] = True
    return m.view(b, T)


def check_fwd(got, x, scale, cu=None):
    out, fin, _ = got
    ro, rf = oracle_fwd(x, scale, cu)
    m = inside(x, cu)
    dt = "f32" if x["q"].dtype == torch.float32 else "bf16"
    if m.any():
        assert_close(out.cpu()[m], ro[m.numpy()], dt, "out")
    if rf.size:
        within(fin, rf, TOL_STATE[dt], "states")


def check_bwd(got, x, dout, dfin, scale, cu=None):
    ref = oracle_bwd(x, dout, dfin, scale, cu)
    dt = "f32" if x["q"].dtype == torch.float32 else "bf16"
    gates = "f32" if x["g"].dtype == torch.float32 else "bf16"
    outside = ~inside(x, cu)
    for n in ("q", "k", "v", "g", "beta"):
        assert got[n].shape == x[n].shape and got[n].dtype == x[n].dtype
        assert not f64(got[n].cpu()[outside]).any(), n
        if dt == "f32":
            within(got[n], ref[n], 1e-4, n)
        elif n in ("g", "beta") and gates == "f32":
            within(got[n], ref[n], TOL_GATE[dt], n)
        else:
            assert_close(got[n], ref[n], "bf16", n)
    if x["initial_states"] is None:
        assert got["initial_states"] is None
    else:
        within(got["initial_states"], ref["init"], TOL_GATE[dt], "initial_states")
