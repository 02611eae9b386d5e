"""tests/delta_device.py is the oracle's recurrence (CPU)."""
import pytest
import torch

from oracle import delta
from tests.delta_cases import draw, draw_grads
from tests.delta_device import rule
from tests.helpers import rel_l2


@pytest.mark.parametrize("b,cu", [(3, None), (1, [2, 2, 9, 20])])
@pytest.mark.parametrize("init", [False, True])
def test_is_the_oracle(b, cu, init):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32)
    x = draw(b, 24, 4, 2, 16, 32, "f32", init=init, nseq=None if cu is None else len(cu) - 1)
    dout, dfin = draw_grads(x)
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"])
    out, final, got = rule(x, 0.3, c, dout, dfin)
    ro, rf, _, _ = delta.delta_fwd(*args, 0.3, x["initial_states"], c)
    ref = delta.delta_bwd(*args, dout, 0.3, x["initial_states"], c, dfin)
    inside = ~torch.from_numpy(ro).isnan()
    assert not out[~inside].any() and rel_l2(out[inside], ro[inside.numpy()]) < 1e-13
    assert rel_l2(final, rf) < 1e-13
    for n in ref:
        assert rel_l2(got[n], ref[n]) < 1e-13, n
