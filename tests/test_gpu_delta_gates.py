"""Gradients of bf16 gates over many tokens (more than 65536 tokens times heads, whose backward
keeps the states rounded) where keys are alike and nothing or little decays."""
import numpy as np
import pytest
import torch

from oracle import delta
from state_space_model_ssd_amd import binding
from tests.delta_cases import dev, draw, unit
from tests.helpers import f64

pytestmark = pytest.mark.gpu

RMS = 2.0 ** -8 / 3 ** 0.5        # of one rounding to bf16: at most half a step, 2^-8, evenly spread
SCALE = 64 ** -0.5


def make(kind):
    """Keys about the same (or the same), beta 0.9 to 1, no decay; beta 1 with decay; or neither."""
    x = draw(1, 2112, 32, 4, 32, 64, "bf16", "bf16", init=False, seed=12)
    assert x["g"].numel() > 65536
    r = torch.Generator().manual_seed(13)
    if "alike" in kind or "same" in kind:
        spread = 0.02 * torch.randn(x["k"].shape, generator=r) if "alike" in kind else 0.0
        x["k"] = unit(x["k"][:, :1].float() + spread).to(x["k"].dtype).expand_as(x["k"]).contiguous()
    if "keep" in kind:
        x["g"].zero_()
    x["beta"].copy_(1.0 if "one" in kind else 0.9 + 0.1 * x["beta"].float() if "high" in kind else
                    0.05 + 0.95 * x["beta"].float())
    dout = torch.randn(x["v"].shape, generator=r).to(x["v"].dtype)
    return x, dout


KINDS = ["spread", "keep one", "alike keep high", "alike keep one", "alike one", "same keep one"]


@pytest.mark.parametrize("kind", KINDS)
def test_beta(kind):
    """dbeta is the sum over the values of dR r, of which each is rounded to bf16 once, and rounded
    itself; the products' errors are independent, so their squares add up."""
    x, dout = make(kind)
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"])
    ref = delta.delta_bwd(*args, dout, SCALE)
    beta = f64(x["beta"])[..., None]
    terms = ref["v"] / beta * (delta.delta_fwd(*args, SCALE)[2] / beta)
    assert np.allclose(terms.sum(-1), ref["beta"])
    got = binding.delta_bwd(**dev(x), dout=dout.cuda())
    size = np.linalg.norm(ref["beta"])
    bound = RMS * (2 * np.linalg.norm(terms) ** 2 + size ** 2) ** 0.5
    err = np.linalg.norm(f64(got["beta"]) - ref["beta"])
    print(f"  dbeta: error {err:.3e}, bound {bound:.3e}, of {size:.3e}", flush=True)
    assert err <= bound
