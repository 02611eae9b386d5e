"""Thin Python binding of the C ABI in include/ssd.h (argument marshalling only).

Every stage of the SSD forward runs in the HIP kernels of libssd_hip.so;
this module only checks tensor metadata, allocates outputs and the workspace
with torch (device memory) and passes raw pointers plus the current HIP
stream.  If the library is not built, every call raises: there is no
fallback of any kind.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssd_hip.so")

SSD_OK, SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_WORKSPACE, SSD_ERR_HIP, \
    SSD_ERR_TOO_LARGE = range(6)
NOALLOC_SCRATCH_BYTES = 64 << 20     # SSD_NOALLOC_SCRATCH_BYTES of include/ssd.h
SSD_F32, SSD_BF16 = 0, 1
STAGE_PLAN, STAGE_CUMSUM, STAGE_BMM, STAGE_CHUNK_STATE, STAGE_STATE_PASSING, STAGE_CHUNK_SCAN = \
    (1 << i for i in range(6))
STAGE_ALL = 0x3F
STAGES = {"plan": STAGE_PLAN, "chunk_cumsum": STAGE_CUMSUM, "bmm_chunk": STAGE_BMM,
          "chunk_state": STAGE_CHUNK_STATE, "state_passing": STAGE_STATE_PASSING,
          "chunk_scan": STAGE_CHUNK_SCAN}

EXPORTED = ("ssd_fwd_workspace_size", "ssd_workspace_layout", "ssd_config_supported",
            "ssd_fwd", "ssd_fwd_stages", "ssd_fwd_tuned", "ssd_bwd_workspace_size", "ssd_bwd",
            "ssd_bwd_after_fwd", "ssd_fwd_choices", "ssd_fwd_noalloc", "ssd_gated_norm_fwd",
            "ssd_gated_norm_bwd_workspace_size", "ssd_gated_norm_bwd", "ssd_fwd_gated",
            "ssd_conv_fwd", "ssd_conv_bwd_workspace_size", "ssd_conv_bwd", "ssd_conv_step",
            "ssd_step", "ssd_block_norm_fwd", "ssd_block_norm_bwd_workspace_size",
            "ssd_block_norm_bwd", "ssd_delta_fwd_workspace_size", "ssd_delta_fwd",
            "ssd_delta_bwd_workspace_size", "ssd_delta_bwd", "ssd_delta_step", "ssd_qk_norm_fwd",
            "ssd_qk_norm_bwd_workspace_size", "ssd_qk_norm_bwd", "ssd_status_string")


class SsdError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"ssd: {msg} (status {code})")
        self.code = code


class ProblemC(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk_size", ctypes.c_int64), ("nseq", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("dt_min", ctypes.c_float),
                ("dt_max", ctypes.c_float)]


class LayoutC(ctypes.Structure):
    _fields_ = [("max_chunks", ctypes.c_int64), ("chunk_table", ctypes.c_size_t),
                ("seq_chunks", ctypes.c_size_t), ("delta", ctypes.c_size_t),
                ("dA_cumsum", ctypes.c_size_t), ("cb", ctypes.c_size_t),
                ("chunk_states", ctypes.c_size_t), ("states_in", ctypes.c_size_t),
                ("block_states", ctypes.c_size_t), ("block_logdecay", ctypes.c_size_t),
                ("sync", ctypes.c_size_t),
                ("sp_blocks", ctypes.c_int64), ("total_bytes", ctypes.c_size_t)]


class NormProblemC(ctypes.Structure):
    """ssd_norm_problem_t: the gated RMS norm after the SSD."""
    _fields_ = [("tokens", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("group_size", ctypes.c_int64), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class GateC(ctypes.Structure):
    """ssd_gate_t: the gated RMS norm ssd_fwd_gated applies to its output."""
    _fields_ = [("z", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("group_size", ctypes.c_int64)]


class ConvProblemC(ctypes.Structure):
    """ssd_conv_problem_t: the short causal convolution in front of the SSD."""
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nseq", ctypes.c_int64),
                ("channels_x", ctypes.c_int64), ("channels_b", ctypes.c_int64),
                ("channels_c", ctypes.c_int64), ("width", ctypes.c_int64),
                ("in_stride", ctypes.c_int64), ("din_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("clear_outside", ctypes.c_int32)]


class StepProblemC(ctypes.Structure):
    """ssd_step_problem_t: one token per sequence."""
    _fields_ = [("batch", ctypes.c_int64), ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("nslots", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("dt_dtype", ctypes.c_int32),
                ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


class BlockNormProblemC(ctypes.Structure):
    """ssd_block_norm_problem_t: the norms around a block."""
    _fields_ = [("tokens", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32),
                ("gate_activation", ctypes.c_int32), ("residual_scale", ctypes.c_float),
                ("eps", ctypes.c_float)]


class DeltaProblemC(ctypes.Structure):
    """ssd_delta_problem_t: the gated delta rule over whole prompts."""
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("ngroups", ctypes.c_int64), ("nseq", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("gate_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("clear_outside", ctypes.c_int32)]


class DeltaStepProblemC(ctypes.Structure):
    """ssd_delta_step_problem_t: the gated delta rule, one token per sequence."""
    _fields_ = [("batch", ctypes.c_int64), ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("nslots", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("g_stride", ctypes.c_int64),
                ("beta_stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("gate_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class QkNormProblemC(ctypes.Structure):
    """ssd_qk_norm_problem_t: the norm of queries and keys, with the rotation."""
    _fields_ = [("tokens", ctypes.c_int64), ("q_heads", ctypes.c_int64), ("k_heads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("rotary_pairs", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("dq_stride", ctypes.c_int64), ("dk_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float)]


class TuningC(ctypes.Structure):
    """ssd_tuning_t: pinned kernel choices, 0 = the library's own."""
    _fields_ = [("scan_kernel", ctypes.c_int32), ("sp_vec", ctypes.c_int32),
                ("front", ctypes.c_int32), ("sp_blocks", ctypes.c_int32),
                ("fused", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libssd_hip.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"HIP library {path} is missing; build it with "
            "`python -m state_space_model_ssd_amd.build` (no fallback exists)")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    PP = ctypes.POINTER(ProblemC)
    lib.ssd_fwd_workspace_size.argtypes = [PP]
    lib.ssd_fwd_workspace_size.restype = sz
    lib.ssd_workspace_layout.argtypes = [PP, ctypes.POINTER(LayoutC)]
    lib.ssd_workspace_layout.restype = ctypes.c_int
    lib.ssd_config_supported.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_int64]
    lib.ssd_config_supported.restype = ctypes.c_int
    lib.ssd_fwd.argtypes = [PP] + [vp] * 12 + [vp, sz, vp]
    lib.ssd_fwd.restype = ctypes.c_int
    lib.ssd_fwd_stages.argtypes = [PP] + [vp] * 12 + [vp, sz, ctypes.c_uint32, vp]
    lib.ssd_fwd_stages.restype = ctypes.c_int
    lib.ssd_fwd_tuned.argtypes = [PP] + [vp] * 12 + [vp, sz, ctypes.c_uint32,
                                                     ctypes.POINTER(TuningC), vp]
    lib.ssd_fwd_tuned.restype = ctypes.c_int
    lib.ssd_bwd_workspace_size.argtypes = [PP]
    lib.ssd_bwd_workspace_size.restype = sz
    lib.ssd_bwd.argtypes = [PP] + [vp] * 20 + [vp, sz, vp]
    lib.ssd_bwd.restype = ctypes.c_int
    lib.ssd_bwd_after_fwd.argtypes = [PP] + [vp] * 20 + [vp, sz, vp]
    lib.ssd_bwd_after_fwd.restype = ctypes.c_int
    NP = ctypes.POINTER(NormProblemC)
    lib.ssd_gated_norm_fwd.argtypes = [NP] + [vp] * 5 + [vp]
    lib.ssd_gated_norm_fwd.restype = ctypes.c_int
    lib.ssd_gated_norm_bwd_workspace_size.argtypes = [NP]
    lib.ssd_gated_norm_bwd_workspace_size.restype = sz
    lib.ssd_gated_norm_bwd.argtypes = [NP] + [vp] * 8 + [sz, vp]
    lib.ssd_gated_norm_bwd.restype = ctypes.c_int
    lib.ssd_fwd_gated.argtypes = [PP] + [vp] * 10 + [ctypes.POINTER(GateC), vp, vp, vp, sz, vp]
    lib.ssd_fwd_gated.restype = ctypes.c_int
    lib.ssd_fwd_noalloc.argtypes = [PP] + [vp] * 12 + [vp]
    lib.ssd_fwd_noalloc.restype = ctypes.c_int
    lib.ssd_fwd_choices.argtypes = [PP, ctypes.POINTER(TuningC)]
    lib.ssd_fwd_choices.restype = ctypes.c_int
    CP, SP, BP = (ctypes.POINTER(s) for s in (ConvProblemC, StepProblemC, BlockNormProblemC))
    lib.ssd_conv_fwd.argtypes = [CP] + [vp] * 10
    lib.ssd_conv_bwd_workspace_size.argtypes = [CP]
    lib.ssd_conv_bwd_workspace_size.restype = sz
    lib.ssd_conv_bwd.argtypes = [CP] + [vp] * 13 + [vp, sz, vp]
    lib.ssd_conv_step.argtypes = [CP] + [vp] * 4 + [ctypes.c_int64] + [vp] * 5
    lib.ssd_step.argtypes = [SP] + [vp] * 11
    lib.ssd_block_norm_fwd.argtypes = [BP] + [vp] * 9
    lib.ssd_block_norm_bwd_workspace_size.argtypes = [BP]
    lib.ssd_block_norm_bwd_workspace_size.restype = sz
    lib.ssd_block_norm_bwd.argtypes = [BP] + [vp] * 14 + [vp, sz, vp]
    DP, DSP, QP = (ctypes.POINTER(s) for s in (DeltaProblemC, DeltaStepProblemC, QkNormProblemC))
    lib.ssd_delta_fwd_workspace_size.argtypes = [DP]
    lib.ssd_delta_fwd.argtypes = [DP] + [vp] * 9 + [vp, sz, vp]
    lib.ssd_delta_bwd_workspace_size.argtypes = [DP]
    lib.ssd_delta_bwd.argtypes = [DP] + [vp] * 15 + [vp, sz, vp]
    lib.ssd_delta_step.argtypes = [DSP] + [vp] * 9
    lib.ssd_qk_norm_fwd.argtypes = [QP] + [vp] * 9
    lib.ssd_qk_norm_bwd_workspace_size.argtypes = [QP]
    lib.ssd_qk_norm_bwd.argtypes = [QP] + [vp] * 12 + [vp, sz, vp]
    for fn in (lib.ssd_delta_fwd_workspace_size, lib.ssd_delta_bwd_workspace_size,
               lib.ssd_qk_norm_bwd_workspace_size):
        fn.restype = sz
    for fn in (lib.ssd_conv_fwd, lib.ssd_conv_bwd, lib.ssd_conv_step, lib.ssd_step,
               lib.ssd_block_norm_fwd, lib.ssd_block_norm_bwd, lib.ssd_delta_fwd, lib.ssd_delta_bwd,
               lib.ssd_delta_step, lib.ssd_qk_norm_fwd, lib.ssd_qk_norm_bwd):
        fn.restype = ctypes.c_int
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().ssd_status_string(code).decode()


def _check(code: int):
    if code != SSD_OK:
        raise SsdError(code, status_string(code))


def make_problem(batch, seqlen, nheads, headdim, dstate, ngroups, chunk_size, dtype,
                 nseq=0, dt_min=0.0, dt_max=math.inf) -> ProblemC:
    if isinstance(dtype, torch.dtype):
        dtype = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}.get(dtype, -1)
    return ProblemC(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate),
                    int(ngroups), int(chunk_size), int(nseq), int(dtype), float(dt_min),
                    float(dt_max))


def workspace_size(prob: ProblemC) -> int:
    return int(load_library().ssd_fwd_workspace_size(ctypes.byref(prob)))


def workspace_layout(prob: ProblemC) -> LayoutC:
    lay = LayoutC()
    _check(load_library().ssd_workspace_layout(ctypes.byref(prob), ctypes.byref(lay)))
    return lay


def config_supported(dtype, headdim, dstate, chunk_size) -> bool:
    if isinstance(dtype, torch.dtype):
        dtype = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}.get(dtype, -1)
    return bool(load_library().ssd_config_supported(int(dtype), int(headdim), int(dstate),
                                                    int(chunk_size)))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, dtype, shape, device):
    if t is None:
        return
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def ssd_fwd(x, dt, A, B, C, chunk_size, D=None, dt_bias=None, initial_states=None,
            cu_seqlens=None, seq_idx=None, dt_min=0.0, dt_max=math.inf, out=None,
            final_states=None, return_final_states=True, workspace=None,
            stages: int = STAGE_ALL, tuning="config"):
    """SSD forward on the GPU through the C ABI.

    x (b, T, H, P) fp32|bf16; dt (b, T, H) fp32; A (H) fp32; B, C (b, T, G, N)
    in x's dtype; D, dt_bias (H) fp32 or None; initial_states (nstates, H, P, N)
    fp32 or None; cu_seqlens (nseq + 1) / seq_idx (T) int32 for a packed batch
    (b == 1).  Returns (out, final_states, workspace).

    tuning: "config" looks the shape up in the tuned config file (see
    tuning.py) and keeps the library's own choices for shapes it does not
    list; None keeps the library's choices; a dict with any of scan_kernel,
    sp_vec, front pins them (ssd_tuning_t in include/ssd.h).
    """
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("ssd_fwd runs on the GPU only; x is on " + str(dev))
    nseq = 0
    if cu_seqlens is not None:
        nseq = cu_seqlens.numel() - 1
    elif seq_idx is not None:
        raise ValueError("pass nseq through cu_seqlens, or use ssd_fwd_seq_idx")
    return _run(x, dt, A, B, C, chunk_size, D, dt_bias, initial_states, cu_seqlens, None, nseq,
                dt_min, dt_max, out, final_states, return_final_states, workspace, stages,
                tuning)


def bwd_workspace_size(prob: ProblemC) -> int:
    return int(load_library().ssd_bwd_workspace_size(ctypes.byref(prob)))


def ssd_bwd(x, dt, A, B, C, chunk_size, dout, dfinal_states=None, D=None, dt_bias=None,
            initial_states=None, cu_seqlens=None, dt_min=0.0, dt_max=math.inf, workspace=None,
            after_fwd=False):
    """SSD backward on the GPU through the C ABI: gradients of
    sum(out * dout) + sum(final_states * dfinal_states) for the inputs of
    ssd_fwd (same arguments).  Returns a dict with x, dt, A, B, C, D,
    dt_bias, initial_states (gradients; D, dt_bias and initial_states always
    computed) and the workspace.

    after_fwd: call ssd_bwd_after_fwd, which reuses the forward's
    intermediates left in `workspace` (required, ssd_bwd_workspace_size
    bytes) by an ssd_fwd call on the same inputs."""
    lib = load_library()
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("ssd_bwd runs on the GPU only; x is on " + str(dev))
    f32 = torch.float32
    nseq = cu_seqlens.numel() - 1 if cu_seqlens is not None else 0
    nstates = nseq if nseq > 0 else b
    _need(x, "x", x.dtype, (b, T, H, P), dev)
    _need(dt, "dt", f32, (b, T, H), dev)
    _need(A, "A", f32, (H,), dev)
    _need(B, "B", x.dtype, (b, T, G, N), dev)
    _need(C, "C", x.dtype, (b, T, G, N), dev)
    _need(D, "D", f32, (H,), dev)
    _need(dt_bias, "dt_bias", f32, (H,), dev)
    _need(initial_states, "initial_states", f32, (nstates, H, P, N), dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), dev)
    _need(dout, "dout", x.dtype, (b, T, H, P), dev)
    _need(dfinal_states, "dfinal_states", f32, (nstates, H, P, N), dev)
    prob = make_problem(b, T, H, P, N, G, chunk_size, x.dtype, nseq, dt_min, dt_max)
    # every token lies in a sequence (cu_seqlens runs from 0 to T), so the
    # library writes every entry of these
    g = {"x": torch.empty_like(x), "dt": torch.empty_like(dt), "A": torch.empty(H, dtype=f32, device=dev),
         "B": torch.empty_like(B), "C": torch.empty_like(C), "D": torch.empty(H, dtype=f32, device=dev),
         "dt_bias": torch.empty(H, dtype=f32, device=dev),
         "initial_states": torch.empty((nstates, H, P, N), dtype=f32, device=dev)}
    need = lib.ssd_bwd_workspace_size(ctypes.byref(prob))
    if workspace is None:
        if after_fwd:
            raise ValueError("after_fwd needs the workspace the forward ran with")
        workspace = torch.empty(max(int(need), 256), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        fn = lib.ssd_bwd_after_fwd if after_fwd else lib.ssd_bwd
        code = fn(ctypes.byref(prob), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B),
                           _ptr(C), _ptr(D), _ptr(initial_states), _ptr(cu_seqlens), None,
                           _ptr(dout), _ptr(dfinal_states), _ptr(g["x"]), _ptr(g["dt"]),
                           _ptr(g["A"]), _ptr(g["B"]), _ptr(g["C"]), _ptr(g["D"]),
                           _ptr(g["dt_bias"]), _ptr(g["initial_states"]), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), stream)
    _check(code)
    g["workspace"] = workspace
    return g


def ssd_fwd_seq_idx(x, dt, A, B, C, chunk_size, seq_idx, nseq, **kw):
    """As ssd_fwd for a packed batch described by per-token sequence ids."""
    return _run(x, dt, A, B, C, chunk_size, kw.get("D"), kw.get("dt_bias"),
                kw.get("initial_states"), None, seq_idx, int(nseq), kw.get("dt_min", 0.0),
                kw.get("dt_max", math.inf), kw.get("out"), kw.get("final_states"),
                kw.get("return_final_states", True), kw.get("workspace"),
                kw.get("stages", STAGE_ALL), kw.get("tuning", "config"))


def ssd_fwd_noalloc(x, dt, A, B, C, chunk_size, out, final_states=None, D=None, dt_bias=None,
                    initial_states=None, cu_seqlens=None, seq_idx=None, nseq=0, dt_min=0.0,
                    dt_max=math.inf):
    """The forward through ssd_fwd_noalloc: the library's static scratch array
    is the workspace, and the caller passes the outputs (`out`, and
    `final_states` or None), so nothing is allocated here either.  For a
    packed batch pass cu_seqlens, or seq_idx with nseq."""
    lib = load_library()
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    f32 = torch.float32
    if dev.type != "cuda":
        raise ValueError("ssd_fwd_noalloc runs on the GPU only; x is on " + str(dev))
    if cu_seqlens is not None:
        nseq = cu_seqlens.numel() - 1
    nstates = nseq if nseq > 0 else b
    for t, name, dtp, shape in ((x, "x", x.dtype, (b, T, H, P)), (dt, "dt", f32, (b, T, H)),
                                (A, "A", f32, (H,)), (B, "B", x.dtype, (b, T, G, N)),
                                (C, "C", x.dtype, (b, T, G, N)), (D, "D", f32, (H,)),
                                (dt_bias, "dt_bias", f32, (H,)),
                                (initial_states, "initial_states", f32, (nstates, H, P, N)),
                                (cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,)),
                                (seq_idx, "seq_idx", torch.int32, (T,)),
                                (out, "out", x.dtype, (b, T, H, P)),
                                (final_states, "final_states", f32, (nstates, H, P, N))):
        _need(t, name, dtp, shape, dev)
    prob = make_problem(b, T, H, P, N, G, chunk_size, x.dtype, nseq, dt_min, dt_max)
    with torch.cuda.device(dev):
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        code = lib.ssd_fwd_noalloc(ctypes.byref(prob), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A),
                                   _ptr(B), _ptr(C), _ptr(D), _ptr(initial_states),
                                   _ptr(cu_seqlens), _ptr(seq_idx), _ptr(out),
                                   _ptr(final_states), stream)
    _check(code)
    return out, final_states


def _norm_problem(y, group_size, eps):
    dtype = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}.get(y.dtype, -1)
    C = y.shape[-1]
    return NormProblemC(int(y.numel() // max(C, 1)), int(C), int(group_size), int(dtype),
                        float(eps))


def gated_norm_fwd(y, z, w, group_size, eps=1e-5, out=None, return_rstd=False):
    """ssd_gated_norm_fwd: rmsnorm(y * silu(z)) * w over groups of group_size
    consecutive channels of the last axis.  y, z: (..., channels) in fp32 or
    bf16 on the GPU, w: (channels,) fp32.  out may be y (in place).  Returns
    out, or (out, rstd) with rstd (rows, channels // group_size) fp32."""
    lib = load_library()
    dev = y.device
    if dev.type != "cuda":
        raise ValueError("gated_norm_fwd runs on the GPU only; y is on " + str(dev))
    C = y.shape[-1]
    _need(y, "y", y.dtype, tuple(y.shape), dev)
    _need(z, "z", y.dtype, tuple(y.shape), dev)
    _need(w, "w", torch.float32, (C,), dev)
    if out is None:
        out = torch.empty_like(y)
    _need(out, "out", y.dtype, tuple(y.shape), dev)
    p = _norm_problem(y, group_size, eps)
    rstd = None
    if return_rstd:
        rstd = torch.empty((p.tokens, C // max(int(group_size), 1)), dtype=torch.float32,
                           device=dev)
    with torch.cuda.device(dev):
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        code = lib.ssd_gated_norm_fwd(ctypes.byref(p), _ptr(y), _ptr(z), _ptr(w), _ptr(out),
                                      _ptr(rstd), stream)
    _check(code)
    return (out, rstd) if return_rstd else out


def gated_norm_bwd(y, z, w, dout, group_size, eps=1e-5, workspace=None):
    """ssd_gated_norm_bwd: (dy, dz, dw) of sum(gated_norm_fwd(y, z, w) * dout)."""
    lib = load_library()
    dev = y.device
    if dev.type != "cuda":
        raise ValueError("gated_norm_bwd runs on the GPU only; y is on " + str(dev))
    C = y.shape[-1]
    for t, name in ((y, "y"), (z, "z"), (dout, "dout")):
        _need(t, name, y.dtype, tuple(y.shape), dev)
    _need(w, "w", torch.float32, (C,), dev)
    p = _norm_problem(y, group_size, eps)
    dy, dz = torch.empty_like(y), torch.empty_like(y)
    dw = torch.empty(C, dtype=torch.float32, device=dev)
    need = int(lib.ssd_gated_norm_bwd_workspace_size(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        code = lib.ssd_gated_norm_bwd(ctypes.byref(p), _ptr(y), _ptr(z), _ptr(w), _ptr(dout),
                                      _ptr(dy), _ptr(dz), _ptr(dw), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), stream)
    _check(code)
    return dy, dz, dw


def ssd_fwd_gated(x, dt, A, B, C, chunk_size, z, norm_weight, group_size, eps=1e-5, D=None,
                  dt_bias=None, initial_states=None, cu_seqlens=None, out=None,
                  final_states=None, workspace=None):
    """ssd_fwd_gated: the forward, then rmsnorm(y * silu(z)) * norm_weight over
    groups of group_size channels of each token's nheads * headdim channels.
    Returns (out, final_states, workspace) like ssd_fwd, out being the
    normalised output."""
    lib = load_library()
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("ssd_fwd_gated runs on the GPU only; x is on " + str(dev))
    f32 = torch.float32
    nseq = cu_seqlens.numel() - 1 if cu_seqlens is not None else 0
    nstates = nseq if nseq > 0 else b
    for t, name, dtp, shape in ((x, "x", x.dtype, (b, T, H, P)), (dt, "dt", f32, (b, T, H)),
                                (A, "A", f32, (H,)), (B, "B", x.dtype, (b, T, G, N)),
                                (C, "C", x.dtype, (b, T, G, N)), (D, "D", f32, (H,)),
                                (dt_bias, "dt_bias", f32, (H,)),
                                (initial_states, "initial_states", f32, (nstates, H, P, N)),
                                (cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,)),
                                (z, "z", x.dtype, (b, T, H, P)),
                                (norm_weight, "norm_weight", f32, (H * P,))):
        _need(t, name, dtp, shape, dev)
    prob = make_problem(b, T, H, P, N, G, chunk_size, x.dtype, nseq)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", x.dtype, (b, T, H, P), dev)
    if final_states is None:
        final_states = torch.empty((nstates, H, P, N), dtype=f32, device=dev)
    _need(final_states, "final_states", f32, (nstates, H, P, N), dev)
    need = lib.ssd_fwd_workspace_size(ctypes.byref(prob))
    if workspace is None:
        workspace = torch.empty(max(int(need), 256), dtype=torch.uint8, device=dev)
    gate = GateC(_ptr(z), _ptr(norm_weight), float(eps), int(group_size))
    with torch.cuda.device(dev):
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        code = lib.ssd_fwd_gated(ctypes.byref(prob), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A),
                                 _ptr(B), _ptr(C), _ptr(D), _ptr(initial_states), _ptr(cu_seqlens),
                                 None, ctypes.byref(gate), _ptr(out), _ptr(final_states),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 stream)
    _check(code)
    return out, final_states, workspace


# ---------------------------------------------------------------------------
# The operators around the scan: short convolution, single-token step, block
# norms.  A decoding step is a few microseconds of GPU time, so these calls
# keep the host's part small: problem structs and workspace sizes are made
# once per set of sizes, and pointers go to ctypes as plain integers.  A tensor
# that a call writes may not share memory with another of its tensors, except
# where a call says so: the library refuses it.
# ---------------------------------------------------------------------------
_DT = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}


@functools.lru_cache(maxsize=1024)
def _conv_problem(*sizes):
    p = ConvProblemC(*sizes)
    return p, ctypes.byref(p), int(load_library().ssd_conv_bwd_workspace_size(ctypes.byref(p)))


@functools.lru_cache(maxsize=1024)
def _step_problem(*sizes):
    p = StepProblemC(*sizes)
    return p, ctypes.byref(p)


@functools.lru_cache(maxsize=1024)
def _block_norm_problem(*sizes):
    p = BlockNormProblemC(*sizes)
    return p, ctypes.byref(p), int(load_library().ssd_block_norm_bwd_workspace_size(ctypes.byref(p)))


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# the current stream's handle without making a torch.cuda.Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(dev, fn, *args):
    """fn(*args, stream) with `dev` current, on its current stream."""
    index = dev.index
    if torch.cuda.current_device() == index:
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _raw_stream(index))
    if code != SSD_OK:
        _check(code)


def _workspace(workspace, need, dev):
    """The caller's workspace (its size and alignment are the library's to
    check), or one made for this call."""
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    return workspace


def _on_gpu(t, name, what):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on the GPU only; {name} is on {dev}")
    if t.dtype not in _DT:
        raise ValueError(f"{name} has dtype {t.dtype}, expected torch.float32 or torch.bfloat16")
    return dev


def _row_stride(t, name, rows):
    """Elements from one row to the next of a tensor whose last axes are
    contiguous and whose first `rows` axes lie evenly behind one another."""
    st, sh = t.stride(), t.shape
    if t.is_contiguous():
        return math.prod(sh[rows:])
    inner = 1
    for i in range(len(sh) - 1, rows - 1, -1):
        if sh[i] != 1 and st[i] != inner:
            raise ValueError(f"{name}'s rows must be contiguous")
        inner *= sh[i]
    # the distance of two rows: of the innermost row axis that has two
    stride = None
    step = 1
    for i in range(rows - 1, -1, -1):
        if sh[i] != 1:
            if stride is None:
                stride = st[i]
                if stride < inner and t.numel() > 0:
                    raise ValueError(f"{name}'s rows overlap")
            elif st[i] != stride * step and t.numel() > 0:
                raise ValueError(f"{name}'s rows must lie evenly behind one another")
            step *= sh[i]
    return inner if stride is None or t.numel() == 0 else stride


_CONV_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}


def _conv_checked(what, x, weight, bias, splits, activation):
    dev = _on_gpu(x, "x", what)
    C = x.shape[-1]
    if weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected ({C}, width)")
    f32 = torch.float32
    _need(weight, "weight", f32, weight.shape, dev)
    _need(bias, "bias", f32, (C,), dev)
    if splits is None:
        splits = (C, 0, 0)
    if len(splits) != 3 or sum(splits) != C:
        raise ValueError(f"splits {tuple(splits)} are not three channel counts with sum {C}")
    if activation not in _CONV_ACTIVATIONS:
        raise ValueError("activation is 'silu' or None")
    return dev, C, tuple(splits), _CONV_ACTIVATIONS[activation]


def _conv_prompt(what, x, weight, bias, splits, activation, initial_states, cu_seqlens, given,
                 dx_stride=0):
    """given: the caller's tensor for what the call writes (None: the call makes it, and
    clears its rows of tokens outside every sequence)."""
    if x.dim() != 3:
        raise ValueError(f"x has {x.dim()} dimensions, expected (batch, seqlen, channels)")
    dev, C, splits, act = _conv_checked(what, x, weight, bias, splits, activation)
    b, T = x.shape[0], x.shape[1]
    nseq = 0
    if cu_seqlens is not None:
        nseq = cu_seqlens.numel() - 1
        if nseq < 1:
            raise ValueError("cu_seqlens needs at least two entries")
        _need(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), dev)
    sshape = (nseq if nseq > 0 else b, weight.shape[1] - 1, C)
    _need(initial_states, "initial_states", x.dtype, sshape, dev)
    prob = _conv_problem(b, T, nseq, *splits, weight.shape[1], _row_stride(x, "x", 2), dx_stride,
                         _DT[x.dtype], act, int(nseq > 0 and given is None))
    return dev, b, T, C, splits, sshape, prob


def _conv_outs(outs, splits, lead, like, name):
    dtype, dev = like.dtype, like.device
    if outs is None:
        return [like.new_empty(lead + (n,)) for n in splits]
    if len(outs) != 3:
        raise ValueError(f"{name} are three tensors")
    for o, n in zip(outs, splits):
        if o is None and n == 0:
            continue
        if o is None:
            raise ValueError(f"{name}: a tensor is missing")
        _need(o, name, dtype, lead + (n,), dev)
    return outs


def conv_fwd(x, weight, bias=None, splits=None, initial_states=None, cu_seqlens=None,
             activation="silu", outs=None, final_states=None, return_final_states=True):
    """ssd_conv_fwd: the short causal convolution that makes x, B and C.

    x (b, T, C) fp32|bf16, its rows contiguous but possibly inside wider ones
    (a slice of the projection's output); weight (C, K) fp32 with K 2..4; bias
    (C) fp32 or None; splits: the channels of x, B and C (default: all C in
    the first output); initial_states (nstates, K - 1, C) in x's dtype or
    None; cu_seqlens (nseq + 1) int32 for a packed batch (b == 1); activation
    'silu' or None.  Returns (x, B, C, final_states): contiguous (b, T,
    splits[i]) tensors, which viewed as (b, T, heads, headdim) and (b, T,
    groups, dstate) are ssd_fwd's inputs, and the states (nstates, K - 1, C)
    that conv_step and a later call's initial_states take (None without
    return_final_states).  Rows of tokens outside every sequence (before cu_seqlens'
    first entry, from its last on) keep what they held in the caller's `outs`, and are
    zeros in outputs that the call makes.  final_states may not be initial_states, nor
    any output share memory with an input."""
    dev, b, T, C, splits, sshape, prob = _conv_prompt("conv_fwd", x, weight, bias, splits,
                                                      activation, initial_states, cu_seqlens, outs)
    outs = _conv_outs(outs, splits, (b, T), x, "outs")
    if final_states is not None:
        _need(final_states, "final_states", x.dtype, sshape, dev)
    elif return_final_states:
        final_states = x.new_empty(sshape)
    _launch(dev, load_library().ssd_conv_fwd, prob[1], x.data_ptr(), weight.data_ptr(), _addr(bias),
            _addr(initial_states), _addr(cu_seqlens), _addr(outs[0]), _addr(outs[1]),
            _addr(outs[2]), _addr(final_states))
    return outs[0], outs[1], outs[2], final_states


def conv_bwd(x, weight, douts, bias=None, splits=None, initial_states=None, cu_seqlens=None,
             activation="silu", dfinal_states=None, dx=None, workspace=None):
    """ssd_conv_bwd: gradients of sum(out_i * douts[i]) + sum(final_states *
    dfinal_states) for conv_fwd's arguments; douts are three tensors like its
    outputs (ssd_bwd's x, B and C gradients).  Returns a dict with x, weight,
    bias (None without a bias), initial_states (None without one) and the
    workspace.  dx: where x's gradient goes, a (b, T, C) tensor that may be a
    slice of a wider one (the gradient of the projection's output).  Rows of tokens
    outside every sequence keep what they held in the caller's dx, and are zeros in
    one that the call makes."""
    stride = 0
    if dx is not None:
        _on_gpu(dx, "dx", "conv_bwd")
        if dx.dtype != x.dtype or dx.shape != x.shape or dx.device != x.device:
            raise ValueError("dx must be like x")
        stride = _row_stride(dx, "dx", 2)
    dev, b, T, C, splits, sshape, prob = _conv_prompt("conv_bwd", x, weight, bias, splits,
                                                      activation, initial_states, cu_seqlens, dx,
                                                      stride)
    if douts is None:
        raise ValueError("douts are three tensors")
    douts = _conv_outs(douts, splits, (b, T), x, "douts")
    _need(dfinal_states, "dfinal_states", x.dtype, sshape, dev)
    f32 = torch.float32
    if dx is None:
        dx = x.new_empty((b, T, C))
    g = {"x": dx, "weight": weight.new_empty(weight.shape),
         "bias": weight.new_empty((C,)) if bias is not None else None,
         "initial_states": x.new_empty(sshape) if initial_states is not None else None}
    workspace = _workspace(workspace, prob[2], dev)
    _launch(dev, load_library().ssd_conv_bwd, prob[1], x.data_ptr(), weight.data_ptr(), _addr(bias),
            _addr(initial_states), _addr(cu_seqlens), _addr(douts[0]), _addr(douts[1]),
            _addr(douts[2]), _addr(dfinal_states), dx.data_ptr(), g["weight"].data_ptr(),
            _addr(g["bias"]), _addr(g["initial_states"]), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    g["workspace"] = workspace
    return g


def conv_step(x, conv_states, weight, bias=None, splits=None, slots=None, activation="silu",
              outs=None):
    """ssd_conv_step: conv_fwd for one new token per sequence, in place on a
    cache of states.  x (batch, C), its rows possibly inside wider ones;
    conv_states (nslots, K - 1, C) in x's dtype, updated; slots (batch) int32:
    each row's slot, rows outside [0, nslots) and rows whose slot an earlier
    row has being padding (None: row b has slot b).  Returns (x, B, C), each
    (batch, splits[i]); padding's rows of `outs` keep what they held (zeros
    where the call makes the outputs)."""
    if x.dim() != 2:
        raise ValueError(f"x has {x.dim()} dimensions, expected (batch, channels)")
    dev, C, splits, act = _conv_checked("conv_step", x, weight, bias, splits, activation)
    b, K = x.shape[0], weight.shape[1]
    nslots = conv_states.shape[0]
    _need(conv_states, "conv_states", x.dtype, (nslots, K - 1, C), dev)
    _need(slots, "slots", torch.int32, (b,), dev)
    if outs is None and slots is not None:
        outs = [torch.zeros((b, n), dtype=x.dtype, device=dev) for n in splits]
    else:
        outs = _conv_outs(outs, splits, (b,), x, "outs")
    prob = _conv_problem(b, 1, 0, *splits, K, _row_stride(x, "x", 1), 0, _DT[x.dtype], act, 0)
    _launch(dev, load_library().ssd_conv_step, prob[1], x.data_ptr(), weight.data_ptr(),
            _addr(bias), conv_states.data_ptr(), nslots, _addr(slots), _addr(outs[0]),
            _addr(outs[1]), _addr(outs[2]))
    return outs[0], outs[1], outs[2]


def ssd_step(x, dt, A, B, C, states, D=None, dt_bias=None, slots=None, dt_min=0.0, dt_max=math.inf,
             out=None):
    """ssd_step: the SSD for one new token per sequence, in place on a cache
    of states.  x (batch, H, P), B and C (batch, G, N) in fp32 or bf16, dt
    (batch, H) in fp32 or x's dtype; each row contiguous but possibly inside a
    wider one.  A, D, dt_bias (H) fp32; states (nslots, H, P, N) fp32, updated
    (ssd_fwd's final_states are such states); slots as for conv_step.  Returns
    out (batch, H, P); padding's rows of it keep what they held (zeros where
    the call makes it)."""
    dev = _on_gpu(x, "x", "ssd_step")
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x is (batch, heads, headdim), B and C (batch, groups, dstate)")
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    f32 = torch.float32
    bc = (b, G, N)
    for t, name, dtp, shape in ((dt, "dt", dt.dtype, (b, H)), (B, "B", x.dtype, bc),
                                (C, "C", x.dtype, bc)):
        if t.device != dev or t.dtype != dtp or t.shape != shape:
            raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected "
                             f"{dtp} {shape} on {dev}")
    if dt.dtype != f32 and dt.dtype != x.dtype:
        raise ValueError(f"dt has dtype {dt.dtype}, expected torch.float32 or {x.dtype}")
    for t, name in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")):
        _need(t, name, f32, (H,), dev)
    nslots = states.shape[0]
    _need(states, "states", f32, (nslots, H, P, N), dev)
    _need(slots, "slots", torch.int32, (b,), dev)
    if out is None:
        make = torch.empty if slots is None else torch.zeros
        out = make((b, H, P), dtype=x.dtype, device=dev)
    _need(out, "out", x.dtype, (b, H, P), dev)
    prob = _step_problem(b, H, P, N, G, nslots, _row_stride(x, "x", 1), _row_stride(dt, "dt", 1),
                         _row_stride(B, "B", 1), _row_stride(C, "C", 1), _DT[x.dtype],
                         _DT[dt.dtype], float(dt_min), float(dt_max))
    _launch(dev, load_library().ssd_step, prob[1], x.data_ptr(), dt.data_ptr(), _addr(dt_bias),
            A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D), states.data_ptr(), _addr(slots),
            out.data_ptr())
    return out


_GATE_ACTIVATIONS = {"linear": 0, "sigmoid": 1, "silu": 2}


def _block_norm_checked(what, x, residual, gate, post_weight, scale, pre_weight, gate_activation,
                        residual_scale, eps, residual_dtype):
    dev = _on_gpu(x, "x", what)
    C = x.shape[-1]
    shape = x.shape
    _need(x, "x", x.dtype, shape, dev)
    if residual is not None:
        residual_dtype = residual.dtype
    elif residual_dtype is None:
        residual_dtype = x.dtype
    if residual_dtype != torch.float32 and residual_dtype != x.dtype:
        raise ValueError(f"residual has dtype {residual_dtype}, expected torch.float32 or {x.dtype}")
    _need(residual, "residual", residual_dtype, shape, dev)
    _need(gate, "gate", x.dtype, shape, dev)
    for t, name in ((post_weight, "post_weight"), (scale, "scale"), (pre_weight, "pre_weight")):
        _need(t, name, torch.float32, (C,), dev)
    if gate_activation not in _GATE_ACTIVATIONS:
        raise ValueError("gate_activation is 'linear', 'sigmoid' or 'silu'")
    prob = _block_norm_problem(x.numel() // max(C, 1), C, _DT[x.dtype], _DT[residual_dtype],
                               _GATE_ACTIVATIONS[gate_activation], float(residual_scale), float(eps))
    return dev, C, shape, residual_dtype, prob


def block_norm_fwd(x, residual, pre_weight, gate=None, gate_activation="sigmoid", post_weight=None,
                   scale=None, residual_scale=1.0, eps=1e-5, out=None, residual_out=None,
                   residual_dtype=None):
    """ssd_block_norm_fwd: from a block's output x and the residual stream, the
    stream after the block, h = residual + residual_scale * scale * p *
    act(gate) with p = rmsnorm(x) * post_weight (x itself without one), and the
    next block's input rmsnorm(h) * pre_weight.  x, gate (..., C) fp32|bf16;
    residual (..., C) in x's dtype or fp32, or None (then h is in
    residual_dtype, default x's); weights (C) fp32.  residual_out may be
    residual and out may be x (in place).  Returns (out, residual_out)."""
    dev, C, shape, rdt, prob = _block_norm_checked(
        "block_norm_fwd", x, residual, gate, post_weight, scale, pre_weight, gate_activation,
        residual_scale, eps, residual_dtype)
    if out is None:
        out = x.new_empty(shape)
    else:
        _need(out, "out", x.dtype, shape, dev)
    if residual_out is None:
        residual_out = x.new_empty(shape, dtype=rdt)
    else:
        _need(residual_out, "residual_out", rdt, shape, dev)
    _launch(dev, load_library().ssd_block_norm_fwd, prob[1], x.data_ptr(), _addr(residual),
            _addr(gate), _addr(post_weight), _addr(scale), pre_weight.data_ptr(), out.data_ptr(),
            residual_out.data_ptr())
    return out, residual_out


def block_norm_bwd(x, residual, pre_weight, dout, dresidual_out=None, gate=None,
                   gate_activation="sigmoid", post_weight=None, scale=None, residual_scale=1.0,
                   eps=1e-5, workspace=None, residual_dtype=None):
    """ssd_block_norm_bwd: gradients of sum(out * dout) + sum(residual_out *
    dresidual_out) for block_norm_fwd's arguments.  Returns a dict with x,
    residual, gate, post_weight, scale, pre_weight (None for an argument that
    is None) and the workspace."""
    dev, C, shape, rdt, prob = _block_norm_checked(
        "block_norm_bwd", x, residual, gate, post_weight, scale, pre_weight, gate_activation,
        residual_scale, eps, residual_dtype)
    _need(dout, "dout", x.dtype, shape, dev)
    _need(dresidual_out, "dresidual_out", rdt, shape, dev)
    g = {"x": x.new_empty(shape),
         "residual": x.new_empty(shape, dtype=rdt) if residual is not None else None,
         "gate": x.new_empty(shape) if gate is not None else None,
         "post_weight": pre_weight.new_empty((C,)) if post_weight is not None else None,
         "scale": pre_weight.new_empty((C,)) if scale is not None else None,
         "pre_weight": pre_weight.new_empty((C,))}
    workspace = _workspace(workspace, prob[2], dev)
    _launch(dev, load_library().ssd_block_norm_bwd, prob[1], x.data_ptr(), _addr(residual),
            _addr(gate), _addr(post_weight), _addr(scale), pre_weight.data_ptr(), dout.data_ptr(),
            _addr(dresidual_out), g["x"].data_ptr(), _addr(g["residual"]), _addr(g["gate"]),
            _addr(g["post_weight"]), _addr(g["scale"]), g["pre_weight"].data_ptr(),
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    g["workspace"] = workspace
    return g


# ---------------------------------------------------------------------------
# The gated delta rule, and the norm of queries and keys in front of it
# ---------------------------------------------------------------------------
def _stride_of(shape, stride, name, rows):
    return _row_stride(torch.empty_strided(shape, stride, device="meta"), name, rows)


# What a call's sizes, strides and types come to; the small calls cost what the host does for
# them, so it is found once for each.
@functools.lru_cache(maxsize=1024)
def _delta_problem(q, k, v, g, beta, nseq, dtype, gate_dtype, scale, clear):
    if len(q) != 4 or len(v) != 4:
        raise ValueError("q and k are (batch, seqlen, groups, dstate), v (batch, seqlen, heads, headdim)")
    b, T, G, N = q
    H, P = v[2], v[3]
    for shape, want, name in ((k, (b, T, G, N), "k"), (v, (b, T, H, P), "v"), (g, (b, T, H), "g"),
                              (beta, (b, T, H), "beta")):
        if shape != want:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected {want}")
    if gate_dtype not in (torch.float32, dtype):
        raise ValueError(f"g has dtype {gate_dtype}, expected torch.float32 or {dtype}")
    p = DeltaProblemC(b, T, H, P, N, G, nseq, _DT[dtype], _DT[gate_dtype],
                      N ** -0.5 if scale is None else scale, int(nseq > 0 and clear))
    ref, lib = ctypes.byref(p), load_library()
    return (p, ref, int(lib.ssd_delta_fwd_workspace_size(ref)), int(lib.ssd_delta_bwd_workspace_size(ref)),
            (nseq if nseq > 0 else b, H, P, N))


@functools.lru_cache(maxsize=1024)
def _delta_step_problem(q, k, v, g, beta, strides, nslots, dtype, gate_dtype, scale):
    if len(q) != 3 or len(v) != 3:
        raise ValueError("q and k are (batch, groups, dstate), v (batch, heads, headdim)")
    b, G, N = q
    H, P = v[1], v[2]
    for shape, want, name in ((k, (b, G, N), "k"), (v, (b, H, P), "v"), (g, (b, H), "g"), (beta, (b, H), "beta")):
        if shape != want:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected {want}")
    if gate_dtype not in (torch.float32, dtype):
        raise ValueError(f"g has dtype {gate_dtype}, expected torch.float32 or {dtype}")
    rows = [_stride_of(t, st, name, 1) for t, st, name in zip((q, k, v, g, beta), strides, ("q", "k", "v", "g", "beta"))]
    p = DeltaStepProblemC(b, H, P, N, G, nslots, *rows, _DT[dtype], _DT[gate_dtype],
                          N ** -0.5 if scale is None else scale)
    return p, ctypes.byref(p), (b, H, P), (nslots, H, P, N), (b,)


@functools.lru_cache(maxsize=1024)
def _qk_norm_problem(q, q_stride, k, k_stride, dtype, R, dq_stride, dk_stride, norm, eps, interleaved):
    if len(q) < 2 or len(k) != len(q) or k[:-2] != q[:-2] or k[-1] != q[-1]:
        raise ValueError("q is (..., heads, headdim), k the same but for its heads")
    if norm not in _QK_NORMS:
        raise ValueError("norm is 'rms' or 'l2'")
    lead, D = tuple(q[:-2]), q[-1]
    if R is not None and (R < 1 or 2 * R > D):
        raise ValueError(f"inv_freq has {R} entries, expected 1 to {D // 2}")
    p = QkNormProblemC(math.prod(lead), q[-2], k[-2], D, R or 0, _stride_of(q, q_stride, "q", len(lead)),
                       _stride_of(k, k_stride, "k", len(lead)), dq_stride, dk_stride, _DT[dtype],
                       _QK_NORMS[norm], int(interleaved), eps)
    ref = ctypes.byref(p)
    return p, ref, int(load_library().ssd_qk_norm_bwd_workspace_size(ref)), lead, (D,)


def _delta_checked(what, q, k, v, g, beta, scale, initial_states, cu_seqlens, clear):
    dev = _on_gpu(q, "q", what)
    for t, name, dtype in ((q, "q", q.dtype), (k, "k", q.dtype), (v, "v", q.dtype), (g, "g", g.dtype),
                           (beta, "beta", g.dtype)):
        if t.device != dev or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {dtype} on {dev}, contiguous")
    nseq = 0
    if cu_seqlens is not None:
        nseq = cu_seqlens.numel() - 1
        if nseq < 1:
            raise ValueError("cu_seqlens needs at least two entries")
        _need(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), dev)
    prob = _delta_problem(q.shape, k.shape, v.shape, g.shape, beta.shape, nseq, q.dtype, g.dtype,
                          None if scale is None else float(scale), clear)
    sshape = prob[4]
    _need(initial_states, "initial_states", torch.float32, sshape, dev)
    return dev, sshape, prob


def delta_fwd(q, k, v, g, beta, scale=None, initial_states=None, cu_seqlens=None, out=None,
              final_states=None, return_final_states=True, workspace=None):
    """ssd_delta_fwd: the gated delta rule over whole prompts.

    q, k (b, T, G, N) and v (b, T, H, P) fp32 or bf16, q and k as qk_norm_fwd
    leaves them; g (log decays) and beta (b, T, H) in fp32 or q's dtype; N 32, 64 or
    128, P a multiple of 16 up to 256; scale: of the output (default N ** -0.5);
    initial_states (nstates, H, P, N) fp32 or None; cu_seqlens (nseq + 1) int32 for a
    packed batch (b == 1).  Returns (out, final_states, workspace): out like v, and the
    states that delta_step and a later call's initial_states take (None without
    return_final_states).  Rows of tokens outside every sequence keep what they held in
    the caller's `out`, and are zeros in one that the call makes."""
    dev, sshape, prob = _delta_checked("delta_fwd", q, k, v, g, beta, scale, initial_states,
                                       cu_seqlens, out is None)
    if out is None:
        out = torch.empty_like(v)
    else:
        _need(out, "out", v.dtype, v.shape, dev)
    if final_states is not None:
        _need(final_states, "final_states", torch.float32, sshape, dev)
    elif return_final_states:
        final_states = v.new_empty(sshape, dtype=torch.float32)
    workspace = _workspace(workspace, prob[2], dev)
    _launch(dev, load_library().ssd_delta_fwd, prob[1], q.data_ptr(), k.data_ptr(), v.data_ptr(),
            g.data_ptr(), beta.data_ptr(), _addr(initial_states), _addr(cu_seqlens), out.data_ptr(),
            _addr(final_states), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, final_states, workspace


def delta_bwd(q, k, v, g, beta, dout, dfinal_states=None, scale=None, initial_states=None,
              cu_seqlens=None, workspace=None):
    """ssd_delta_bwd: gradients of sum(out * dout) + sum(final_states * dfinal_states) for
    delta_fwd's arguments.  Returns a dict with q, k, v, g, beta (each like its argument;
    rows of tokens outside every sequence are zeros), initial_states (None without one) and
    the workspace.  With bf16 g and beta of 65536 tokens times heads or more their gradients come
    from states rounded to bf16 (include/ssd.h says how far off); fp32 ones do not."""
    dev, sshape, prob = _delta_checked("delta_bwd", q, k, v, g, beta, scale, initial_states,
                                       cu_seqlens, True)
    _need(dout, "dout", v.dtype, v.shape, dev)
    _need(dfinal_states, "dfinal_states", torch.float32, sshape, dev)
    if dout is None:
        raise ValueError("dout is missing")
    grads = {"q": torch.empty_like(q), "k": torch.empty_like(k), "v": torch.empty_like(v),
             "g": torch.empty_like(g), "beta": torch.empty_like(beta),
             "initial_states": v.new_empty(sshape, dtype=torch.float32)
             if initial_states is not None else None}
    workspace = _workspace(workspace, prob[3], dev)
    _launch(dev, load_library().ssd_delta_bwd, prob[1], q.data_ptr(), k.data_ptr(), v.data_ptr(),
            g.data_ptr(), beta.data_ptr(), _addr(initial_states), _addr(cu_seqlens), dout.data_ptr(),
            _addr(dfinal_states), grads["q"].data_ptr(), grads["k"].data_ptr(),
            grads["v"].data_ptr(), grads["g"].data_ptr(), grads["beta"].data_ptr(),
            _addr(grads["initial_states"]), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    grads["workspace"] = workspace
    return grads


def delta_step(q, k, v, g, beta, states, scale=None, slots=None, out=None):
    """ssd_delta_step: the gated delta rule for one new token per sequence, in place on a
    cache of states.  q, k (batch, G, N) and v (batch, H, P) fp32 or bf16, g and beta
    (batch, H) in fp32 or q's dtype; each row contiguous but possibly inside a wider one;
    any P, N up to 256.  states (nslots, H, P, N) fp32, updated (delta_fwd's final_states
    are such states); slots as for conv_step.  Returns out (batch, H, P); padding's rows of
    it keep what they held (zeros where the call makes it)."""
    dev = _on_gpu(q, "q", "delta_step")
    for t, name, dtype in ((k, "k", q.dtype), (v, "v", q.dtype), (g, "g", g.dtype), (beta, "beta", g.dtype)):
        if t.device != dev or t.dtype != dtype:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {dtype} on {dev}")
    prob = _delta_step_problem(q.shape, k.shape, v.shape, g.shape, beta.shape,
                               (q.stride(), k.stride(), v.stride(), g.stride(), beta.stride()),
                               states.shape[0], q.dtype, g.dtype, None if scale is None else float(scale))
    _need(states, "states", torch.float32, prob[3], dev)
    _need(slots, "slots", torch.int32, prob[4], dev)
    if out is None:
        make = torch.empty if slots is None else torch.zeros
        out = make(prob[2], dtype=v.dtype, device=dev)
    else:
        _need(out, "out", v.dtype, prob[2], dev)
    _launch(dev, load_library().ssd_delta_step, prob[1], q.data_ptr(), k.data_ptr(), v.data_ptr(),
            g.data_ptr(), beta.data_ptr(), states.data_ptr(), _addr(slots), out.data_ptr())
    return out


_QK_NORMS = {"rms": 0, "l2": 1}


def _qk_norm_checked(what, q, k, q_weight, k_weight, norm, eps, positions, inv_freq, interleaved,
                     dq_stride=0, dk_stride=0):
    dev = _on_gpu(q, "q", what)
    if k.dtype != q.dtype or k.device != dev:
        raise ValueError(f"k is {k.dtype} on {k.device}, expected {q.dtype} on {dev}")
    if (positions is None) != (inv_freq is None):
        raise ValueError("the rotation takes both positions and inv_freq")
    R = None if inv_freq is None else inv_freq.numel()
    prob = _qk_norm_problem(q.shape, q.stride(), k.shape, k.stride(), q.dtype, R, dq_stride, dk_stride,
                            norm, float(eps), bool(interleaved))
    _need(q_weight, "q_weight", torch.float32, prob[4], dev)
    _need(k_weight, "k_weight", torch.float32, prob[4], dev)
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float32, (R,), dev)
        _need(positions, "positions", torch.int32, prob[3], dev)
    return dev, prob


def qk_norm_fwd(q, k, q_weight=None, k_weight=None, norm="rms", eps=1e-6, positions=None,
                inv_freq=None, interleaved=False, outs=None):
    """ssd_qk_norm_fwd: the norm of queries and keys in each head, and the rotation by the
    token's position, in one pass.  q (..., Hq, D), k (..., Hk, D) fp32 or bf16, each
    token's heads contiguous but possibly inside wider rows; weights (D) fp32 or None;
    norm 'rms' (by the mean of squares) or 'l2' (by their sum: unit length, as the gated
    delta rule takes them); positions (...) int32 and inv_freq (R) fp32 turn the first 2 R
    channels, as pairs (i, i + R) or, interleaved, (2i, 2i + 1); None: no rotation.
    Returns contiguous (q, k)."""
    dev, prob = _qk_norm_checked("qk_norm_fwd", q, k, q_weight, k_weight, norm, eps, positions,
                                 inv_freq, interleaved)
    if outs is None:
        outs = (torch.empty_like(q, memory_format=torch.contiguous_format),
                torch.empty_like(k, memory_format=torch.contiguous_format))
    else:
        if len(outs) != 2:
            raise ValueError("outs are two tensors")
        for o, like in zip(outs, (q, k)):
            _need(o, "outs", q.dtype, like.shape, dev)
    _launch(dev, load_library().ssd_qk_norm_fwd, prob[1], q.data_ptr(), k.data_ptr(),
            _addr(q_weight), _addr(k_weight), _addr(positions), _addr(inv_freq), outs[0].data_ptr(),
            outs[1].data_ptr())
    return outs[0], outs[1]


def qk_norm_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, norm="rms", eps=1e-6,
                positions=None, inv_freq=None, interleaved=False, dq=None, dk=None, workspace=None):
    """ssd_qk_norm_bwd: gradients of sum(q_out * dq_out) + sum(k_out * dk_out) for
    qk_norm_fwd's arguments.  Returns a dict with q, k, q_weight, k_weight (None without a
    weight) and the workspace.  dq, dk: where q's and k's gradients go, tensors like q and k
    that may be slices of a wider one (the gradient of the projection's output)."""
    strides = []
    for t, like, name in ((dq, q, "dq"), (dk, k, "dk")):
        if t is not None and (t.dtype != like.dtype or t.shape != like.shape or t.device != like.device):
            raise ValueError(f"{name} must be like {name[1:]}")
        strides.append(0 if t is None else _row_stride(t, name, t.dim() - 2))
    dev, prob = _qk_norm_checked("qk_norm_bwd", q, k, q_weight, k_weight, norm, eps, positions,
                                 inv_freq, interleaved, *strides)
    if dq_out is None or dk_out is None:
        raise ValueError("dq_out and dk_out are the outputs' gradients")
    _need(dq_out, "dq_out", q.dtype, q.shape, dev)
    _need(dk_out, "dk_out", q.dtype, k.shape, dev)
    g = {"q": torch.empty_like(q, memory_format=torch.contiguous_format) if dq is None else dq,
         "k": torch.empty_like(k, memory_format=torch.contiguous_format) if dk is None else dk,
         "q_weight": torch.empty_like(q_weight) if q_weight is not None else None,
         "k_weight": torch.empty_like(k_weight) if k_weight is not None else None}
    need = prob[2] if q_weight is not None or k_weight is not None else 0
    workspace = _workspace(workspace, need, dev)
    _launch(dev, load_library().ssd_qk_norm_bwd, prob[1], q.data_ptr(), k.data_ptr(),
            _addr(q_weight), _addr(k_weight), _addr(positions), _addr(inv_freq), dq_out.data_ptr(),
            dk_out.data_ptr(), g["q"].data_ptr(), g["k"].data_ptr(), _addr(g["q_weight"]),
            _addr(g["k_weight"]), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    g["workspace"] = workspace
    return g


def fwd_choices(prob: ProblemC) -> dict:
    """The library's own kernel choices for this problem on the current
    device (ssd_fwd_choices), as a dict of the ssd_tuning_t fields."""
    t = TuningC(0, 0, 0, 0, 0)
    _check(load_library().ssd_fwd_choices(ctypes.byref(prob), ctypes.byref(t)))
    return {k: int(getattr(t, k)) for k, _ in TuningC._fields_}


def make_tuning(choice) -> TuningC:
    """TuningC from None or a dict of scan_kernel / sp_vec / front / sp_blocks /
    fused."""
    t = TuningC(0, 0, 0, 0, 0)
    if choice:
        unknown = set(choice) - {"scan_kernel", "sp_vec", "front", "sp_blocks", "fused"}
        if unknown:
            raise ValueError(f"unknown tuning fields {sorted(unknown)}")
        for k, v in choice.items():
            setattr(t, k, int(v))
    return t


def _run(x, dt, A, B, C, chunk_size, D, dt_bias, init, cu, sidx, nseq, dt_min, dt_max, out,
         final_states, return_final, workspace, stages, tuning="config"):
    lib = load_library()
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    f32 = torch.float32
    _need(x, "x", x.dtype, (b, T, H, P), dev)
    _need(dt, "dt", f32, (b, T, H), dev)
    _need(A, "A", f32, (H,), dev)
    _need(B, "B", x.dtype, (b, T, G, N), dev)
    _need(C, "C", x.dtype, (b, T, G, N), dev)
    _need(D, "D", f32, (H,), dev)
    _need(dt_bias, "dt_bias", f32, (H,), dev)
    nstates = nseq if nseq > 0 else b
    _need(init, "initial_states", f32, (nstates, H, P, N), dev)
    _need(cu, "cu_seqlens", torch.int32, (nseq + 1,), dev)
    _need(sidx, "seq_idx", torch.int32, (T,), dev)
    prob = make_problem(b, T, H, P, N, G, chunk_size, x.dtype, nseq, dt_min, dt_max)
    if isinstance(tuning, str):
        if tuning != "config":
            raise ValueError("tuning is 'config', None or a dict")
        from state_space_model_ssd_amd import tuning as _tuning
        tuning = _tuning.lookup(prob)
    tune = make_tuning(tuning)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", x.dtype, (b, T, H, P), dev)
    if final_states is None and return_final:
        final_states = torch.empty((nstates, H, P, N), dtype=f32, device=dev)
    _need(final_states, "final_states", f32, (nstates, H, P, N), dev)
    need = lib.ssd_fwd_workspace_size(ctypes.byref(prob))
    if workspace is None:
        workspace = torch.empty(max(int(need), 256), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        stream = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        code = lib.ssd_fwd_tuned(ctypes.byref(prob), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A),
                                 _ptr(B), _ptr(C), _ptr(D), _ptr(init), _ptr(cu), _ptr(sidx),
                                 _ptr(out), _ptr(final_states), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), int(stages),
                                 ctypes.byref(tune), stream)
    _check(code)
    return out, final_states, workspace


def intermediates(workspace: torch.Tensor, prob: ProblemC) -> dict:
    """Views of the stage intermediates inside a workspace (layout of
    ssd_workspace_layout): chunk_table (mc,4), seq_chunks (nstates+1),
    delta/dA_cumsum (mc,H,L), chunk_states (mc,H,P,N) fp32, cb (mc,G,L,L)
    and states_in (mc,H,P,N) in the problem dtype."""
    lay = workspace_layout(prob)
    mc, H, L, G = lay.max_chunks, prob.nheads, prob.chunk_size, prob.ngroups
    P, N = prob.headdim, prob.dstate
    nstates = prob.nseq if prob.nseq > 0 else prob.batch

    def view(off, dtype, shape):
        n = 1
        for s in shape:
            n *= s
        es = torch.tensor([], dtype=dtype).element_size()
        return workspace[off:off + n * es].view(dtype).view(*shape)

    sdt = torch.bfloat16 if prob.dtype == SSD_BF16 else torch.float32
    return dict(
        max_chunks=mc,
        chunk_table=view(lay.chunk_table, torch.int32, (mc, 4)),
        seq_chunks=view(lay.seq_chunks, torch.int32, (nstates + 1,)),
        delta=view(lay.delta, torch.float32, (mc, H, L)),
        dA_cumsum=view(lay.dA_cumsum, torch.float32, (mc, H, L)),
        cb=view(lay.cb, sdt, (mc, G, L, L)),
        chunk_states=view(lay.chunk_states, torch.float32, (mc, H, P, N)),
        states_in=view(lay.states_in, sdt, (mc, H, P, N)),
    )
