"""Refusals of the operators around the SSD beyond tests/test_layer_host.py's (CPU only:
every call fails before anything reaches a device)."""
import ctypes

import pytest

from state_space_model_ssd_amd import binding as b
from tests.test_layer_host import (BAD, UNS, conv, conv_bwd, conv_fwd, conv_step, lib,  # noqa: F401
                                   norm, norm_bwd, norm_fwd, run_step, step)


@pytest.mark.parametrize("value", [-1, 2])
def test_conv_clear_outside_is_a_truth_value(lib, value):  # noqa: F811
    p = conv(clear_outside=value)
    assert conv_fwd(lib, p) == conv_bwd(lib, p) == conv_step(lib, p) == BAD
    assert lib.ssd_conv_bwd_workspace_size(ctypes.byref(p)) == 0
    # without tokens there is nothing to clear, and nothing is launched
    empty = conv(batch=1, seqlen=0, nseq=2, clear_outside=1)
    assert lib.ssd_conv_fwd(ctypes.byref(empty), *[None] * 9, None) == b.SSD_OK


# The limits that include/ssd.h states: the size on them is taken, the next is not.
CONV_LIMITS = [
    (dict(channels_x=2 ** 20 - 32, batch=1), dict(channels_x=2 ** 20 - 31, batch=1)),
    (dict(batch=65535, seqlen=1), dict(batch=65536, seqlen=1)),
    (dict(batch=1, nseq=65535), dict(batch=1, nseq=65536)),
    (dict(batch=1, seqlen=2 ** 30), dict(batch=1, seqlen=2 ** 30 + 1)),
    (dict(batch=32768, seqlen=2 ** 15), dict(batch=32768, seqlen=2 ** 15 + 1)),
    (dict(batch=1, seqlen=2 ** 25, channels_x=2 ** 15, channels_b=0, channels_c=0),
     dict(batch=1, seqlen=2 ** 25, channels_x=2 ** 15 + 1, channels_b=0, channels_c=0)),
    (dict(batch=2 ** 15, channels_x=2 ** 15 - 32), dict(batch=2 ** 15, channels_x=2 ** 15 - 31)),
    (dict(width=2), dict(width=1)), (dict(width=4), dict(width=5)),
]


@pytest.mark.parametrize("on,beyond", CONV_LIMITS)
def test_conv_limits(lib, on, beyond):  # noqa: F811
    assert lib.ssd_conv_bwd_workspace_size(ctypes.byref(conv(**on))) > 0
    assert conv_fwd(lib, conv(**on), x=None) == BAD          # a size that is taken, no input
    assert conv_fwd(lib, conv(**beyond)) == conv_bwd(lib, conv(**beyond)) == UNS
    assert lib.ssd_conv_bwd_workspace_size(ctypes.byref(conv(**beyond))) == 0


STEP_LIMITS = [
    (dict(dstate=256), dict(dstate=257)),
    (dict(batch=65535), dict(batch=65536)),
    (dict(nheads=65535, ngroups=1), dict(nheads=65536, ngroups=1)),
    (dict(headdim=65535), dict(headdim=65536)),
    (dict(nslots=2 ** 31 - 1), dict(nslots=2 ** 31)),
    # 8 rows per workgroup of dstate 128, 4 of 256, 128 of 7, 64 of 9, 256 of 1
    (dict(batch=2 ** 15, nheads=2 ** 5, headdim=64), dict(batch=2 ** 15, nheads=2 ** 5, headdim=65)),
    (dict(batch=2 ** 14, nheads=2 ** 5, headdim=64, dstate=256),
     dict(batch=2 ** 14, nheads=2 ** 5, headdim=65, dstate=256)),
    (dict(batch=2 ** 15, nheads=2 ** 7, headdim=256, dstate=7),
     dict(batch=2 ** 15, nheads=2 ** 7, headdim=257, dstate=7)),
    (dict(batch=2 ** 15, nheads=2 ** 7, headdim=128, dstate=9),
     dict(batch=2 ** 15, nheads=2 ** 7, headdim=129, dstate=9)),
    (dict(batch=2 ** 15, nheads=2 ** 7, headdim=512, dstate=1),
     dict(batch=2 ** 15, nheads=2 ** 7, headdim=513, dstate=1)),
]


@pytest.mark.parametrize("on,beyond", STEP_LIMITS)
def test_step_limits(lib, on, beyond):  # noqa: F811
    base = dict(nslots=70000)
    assert run_step(lib, step(**{**base, **on}), null=("x",)) == BAD
    assert run_step(lib, step(**{**base, **beyond})) == UNS


@pytest.mark.parametrize("on,beyond", [
    (dict(channels=8192), dict(channels=8193)),
    (dict(tokens=2 ** 32, channels=256), dict(tokens=2 ** 32 + 1, channels=256)),
    (dict(tokens=2 ** 40, channels=1), dict(tokens=2 ** 40 + 1, channels=1)),
])
def test_block_norm_limits(lib, on, beyond):  # noqa: F811
    assert lib.ssd_block_norm_bwd_workspace_size(ctypes.byref(norm(**on))) > 0
    assert norm_fwd(lib, norm(**on), x=None) == BAD
    assert norm_fwd(lib, norm(**beyond)) == norm_bwd(lib, norm(**beyond)) == UNS


def test_strides_and_slots(lib):  # noqa: F811
    assert conv_fwd(lib, conv(in_stride=2 ** 31), w=None) == BAD     # taken, no weight
    assert conv_fwd(lib, conv(in_stride=2 ** 31 + 1)) == BAD
    assert conv_bwd(lib, conv(din_stride=2 ** 31), ws=None) == b.SSD_ERR_WORKSPACE
    assert conv_bwd(lib, conv(din_stride=2 ** 31 + 1), ws=None) == BAD
    p = conv(seqlen=1)
    assert conv_step(lib, p, nslots=2 ** 31 - 1, x=None) == BAD
    assert conv_step(lib, p, nslots=2 ** 31, x=None) == UNS
    for k in ("x_stride", "dt_stride", "b_stride", "c_stride"):
        assert run_step(lib, step(**{k: 2 ** 31 + 1})) == BAD
