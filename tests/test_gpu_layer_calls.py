"""Calls of the operators around the SSD that are easy to make by mistake, or that leave
something out (GPU): refused, or answered as documented."""
import pytest
import torch

from state_space_model_ssd_amd import binding

pytestmark = pytest.mark.gpu


def conv_args(T=40, C=24, K=4, b=1, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return r(b, T, C).to(dtype), r(C, K)


def test_conv_backward_without_output_gradients_is_refused():
    x, w = conv_args()
    with pytest.raises(ValueError, match="douts"):
        binding.conv_bwd(x, w, None)
