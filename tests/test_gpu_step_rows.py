"""The single-token state update where a thread has two or four rows and the sizes leave a
remainder (GPU), with padding and repeated slots, against the fp64 oracle within the bounds
of tests/test_gpu_step.py.  The state is updated in place, so states of no row and the
cache's guard states are held to what they were, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import layer
from state_space_model_ssd_amd import binding
from tests.layer_bounds import DT, RND, TINY, check
from tests.step_rows_cases import CASES
from tests.test_gpu_step import bounds, device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", sorted(CASES))
def test_step_with_several_rows_per_thread(name):
    batch, H, P, N, G, dtype, dtd, D, bias = CASES[name][1]
    g = torch.Generator().manual_seed(batch + N)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    nslots = batch + 3
    row = r(batch, H * P + 2 * G * N + 5).to(DT[dtype])
    d = dict(row=row, x=row[:, :H * P].unflatten(1, (H, P)),
             B=row[:, H * P:H * P + G * N].unflatten(1, (G, N)),
             C=row[:, H * P + G * N:H * P + 2 * G * N].unflatten(1, (G, N)),
             dt=(r(batch, H) * 2 - 1).to(DT[dtd]), A=-torch.exp(r(H)), D=r(H) if D else None,
             bias=r(H) if bias else None, states=r(nslots, H, P, N))
    slots = torch.randperm(nslots, generator=g)[:batch].tolist()
    slots[1], slots[-1] = -1, slots[0]              # padding, and a slot that row 0 has
    e = device(d)
    guard = torch.full((nslots + 2, H, P, N), 3.0, device="cuda")
    guard[1:-1] = e["states"]
    st = guard[1:-1]
    out = torch.full((batch, H, P), 5.0, dtype=DT[dtype], device="cuda")
    binding.ssd_step(e["x"], e["dt"], e["A"], e["B"], e["C"], st, D=e["D"], dt_bias=e["bias"],
                     slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert (guard[0] == 3).all() and (guard[-1] == 3).all()
    ref, sref = layer.ssd_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["states"], d["D"], d["bias"],
                               slots)
    se, ye, idx = bounds(d, slots)
    pads = np.array(layer.padding_rows(slots, batch, nslots))
    assert pads.sum() == 2
    tol = np.zeros_like(sref)                      # states that no row has: not touched
    tol[idx[~pads]] = se[~pads]
    check(st, sref, tol, "state")
    assert (out.cpu()[torch.from_numpy(pads)] == 5).all()
    check(out, ref, ye + RND[dtype] * (np.abs(np.nan_to_num(ref)) + ye) + TINY, "out")
