"""Refusals of the operators around the SSD beyond tests/test_layer_host.py's (CPU only:
every call fails before anything reaches a device)."""
import ctypes

import pytest

from state_space_model_ssd_amd import binding as b
from tests.test_layer_host import BAD, conv, conv_bwd, conv_fwd, conv_step, lib  # noqa: F401


@pytest.mark.parametrize("value", [-1, 2])
def test_conv_clear_outside_is_a_truth_value(lib, value):  # noqa: F811
    p = conv(clear_outside=value)
    assert conv_fwd(lib, p) == conv_bwd(lib, p) == conv_step(lib, p) == BAD
    assert lib.ssd_conv_bwd_workspace_size(ctypes.byref(p)) == 0
    # without tokens there is nothing to clear, and nothing is launched
    empty = conv(batch=1, seqlen=0, nseq=2, clear_outside=1)
    assert lib.ssd_conv_fwd(ctypes.byref(empty), *[None] * 9, None) == b.SSD_OK
