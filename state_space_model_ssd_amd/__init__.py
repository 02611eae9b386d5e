"""Mamba-2 SSD chunked-scan forward on AMD Instinct MI355X (gfx950).

The compute path is the HIP library libssd_hip.so (C ABI: include/ssd.h);
`binding` marshals torch tensors into it.  Importing the package does not
load the library; the first call does, and raises if it is not built.
"""
from .binding import (ssd_fwd, ssd_fwd_seq_idx, load_library, workspace_size,  # noqa: F401
                      workspace_layout, intermediates, make_problem, config_supported,
                      conv_fwd, conv_bwd, conv_step, ssd_step, block_norm_fwd, block_norm_bwd,
                      delta_fwd, delta_bwd, delta_step, qk_norm_fwd, qk_norm_bwd,
                      SsdError, STAGES, STAGE_ALL)
