"""Host-side checks of the operators around the SSD (CPU only: every call fails,
or has nothing to launch, before anything reaches a device)."""
import ctypes

import pytest
import torch

from state_space_model_ssd_amd import binding as b

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)
BAD, UNS, WSP = b.SSD_ERR_INVALID_ARG, b.SSD_ERR_UNSUPPORTED, b.SSD_ERR_WORKSPACE
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return b.load_library()


def conv(**kw):
    base = dict(batch=2, seqlen=100, nseq=0, channels_x=64, channels_b=16, channels_c=16, width=4,
                in_stride=0, din_stride=0, dtype=b.SSD_BF16, activation=1)
    base.update(kw)
    return b.ConvProblemC(**base)


def conv_fwd(lib, p, x=FAKE, w=FAKE, init=None, cu=None, outs=(FAKE, FAKE, FAKE), fin=None):
    return lib.ssd_conv_fwd(ctypes.byref(p), x, w, None, init, cu, *outs, fin, None)


def conv_bwd(lib, p, x=FAKE, w=FAKE, cu=None, douts=(FAKE, FAKE, FAKE), dx=FAKE, dw=FAKE, ws=FAKE,
             size=1 << 40):
    return lib.ssd_conv_bwd(ctypes.byref(p), x, w, None, None, cu, *douts, None, dx, dw, None, None,
                            ws, size, None)


def conv_step(lib, p, x=FAKE, states=FAKE, nslots=2, slots=None, outs=(FAKE, FAKE, FAKE)):
    return lib.ssd_conv_step(ctypes.byref(p), x, FAKE, None, states, nslots, slots, *outs, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(seqlen=-1), BAD), (dict(nseq=-1), BAD), (dict(channels_x=0), BAD),
    (dict(channels_b=-1), BAD), (dict(channels_c=-8), BAD), (dict(width=0), BAD),
    (dict(dtype=2), BAD), (dict(activation=2), BAD), (dict(activation=-1), BAD),
    (dict(nseq=3), BAD),                                   # packed needs batch 1
    (dict(in_stride=95), BAD), (dict(in_stride=-96), BAD), (dict(din_stride=1), BAD),
    (dict(width=1), UNS), (dict(width=5), UNS), (dict(channels_x=1 << 21), UNS),
    (dict(channels_x=1 << 62, channels_b=1 << 62, channels_c=1 << 62), UNS),
    (dict(batch=70000), UNS), (dict(seqlen=1 << 31), UNS), (dict(batch=60000, seqlen=1 << 30), UNS),
    (dict(batch=65535, channels_x=1 << 19), UNS),
])
def test_conv_problems_refused(lib, kw, code):
    p = conv(**kw)
    assert conv_fwd(lib, p) == conv_bwd(lib, p) == code
    assert conv_step(lib, p) == code
    assert lib.ssd_conv_bwd_workspace_size(ctypes.byref(p)) == 0


def test_conv_null_problem(lib):
    assert lib.ssd_conv_fwd(None, *[FAKE] * 9, None) == BAD
    assert lib.ssd_conv_bwd_workspace_size(None) == 0


def test_conv_pointers_and_packing(lib):
    p = conv()
    for kw in (dict(x=None), dict(w=None), dict(outs=(None, FAKE, FAKE)), dict(outs=(FAKE, None, FAKE)),
               dict(outs=(FAKE, FAKE, None)), dict(x=ODD), dict(init=ODD), dict(fin=ODD),
               dict(outs=(FAKE, ODD, FAKE)), dict(cu=FAKE)):
        assert conv_fwd(lib, p, **kw) == BAD, kw
    for kw in (dict(x=None), dict(w=None), dict(dw=None), dict(dx=None), dict(dx=ODD),
               dict(douts=(FAKE, FAKE, None)), dict(cu=FAKE)):
        assert conv_bwd(lib, p, **kw) == BAD, kw
    assert conv_fwd(lib, conv(batch=1, nseq=2)) == BAD          # packed without cu_seqlens
    # no tokens and nothing to write: ok without a launch
    empty = conv(batch=1, seqlen=0, nseq=2)
    assert lib.ssd_conv_fwd(ctypes.byref(empty), *[None] * 9, None) == b.SSD_OK
    assert lib.ssd_conv_fwd(ctypes.byref(conv(batch=0)), *[None] * 9, None) == b.SSD_OK


def test_conv_workspace(lib):
    p = conv()
    need = lib.ssd_conv_bwd_workspace_size(ctypes.byref(p))
    assert need > 0 and need % 256 == 0
    assert conv_bwd(lib, p, ws=None) == WSP
    assert conv_bwd(lib, p, size=need - 1) == WSP
    assert conv_bwd(lib, p, ws=ctypes.c_void_p(0x1008)) == WSP


def test_conv_step_arguments(lib):
    p = conv(seqlen=1)
    assert conv_step(lib, conv(seqlen=2)) == BAD
    assert conv_step(lib, conv(batch=1, seqlen=1, nseq=1)) == BAD
    for kw in (dict(nslots=-1), dict(nslots=1), dict(states=None), dict(states=ODD), dict(x=None),
               dict(outs=(FAKE, FAKE, None))):
        assert conv_step(lib, p, **kw) == BAD, kw
    assert conv_step(lib, p, nslots=1 << 40, slots=FAKE) == UNS
    assert conv_step(lib, conv(batch=0, seqlen=1), x=None, states=None, nslots=0) == b.SSD_OK


def step(**kw):
    base = dict(batch=2, nheads=8, headdim=64, dstate=128, ngroups=2, nslots=4, x_stride=0,
                dt_stride=0, b_stride=0, c_stride=0, dtype=b.SSD_BF16, dt_dtype=b.SSD_F32,
                dt_min=0.0, dt_max=INF)
    base.update(kw)
    return b.StepProblemC(**base)


def run_step(lib, p, null=(), odd=(), slots=None):
    ptr = {k: FAKE for k in ("x", "dt", "bias", "A", "B", "C", "D", "states", "out")}
    ptr.update({k: None for k in null})
    ptr.update({k: ODD for k in odd})
    return lib.ssd_step(ctypes.byref(p), ptr["x"], ptr["dt"], ptr["bias"], ptr["A"], ptr["B"],
                        ptr["C"], ptr["D"], ptr["states"], slots, ptr["out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(nheads=0), BAD), (dict(headdim=0), BAD), (dict(dstate=0), BAD),
    (dict(ngroups=0), BAD), (dict(ngroups=3), BAD), (dict(nslots=-1), BAD), (dict(nslots=1), BAD),
    (dict(dtype=2), BAD), (dict(dt_dtype=-1), BAD), (dict(dtype=b.SSD_F32, dt_dtype=b.SSD_BF16), BAD),
    (dict(dt_min=2.0, dt_max=1.0), BAD), (dict(dt_min=NAN), BAD), (dict(dt_max=NAN), BAD),
    (dict(x_stride=511), BAD), (dict(dt_stride=7), BAD), (dict(b_stride=255), BAD),
    (dict(c_stride=-1), BAD),
    (dict(dstate=257), UNS), (dict(batch=65536, nslots=65536), UNS), (dict(headdim=1 << 40), UNS),
    (dict(nheads=1 << 40, ngroups=1), UNS), (dict(nslots=1 << 40), UNS),
    (dict(batch=65535, nslots=65535, nheads=1024), UNS),
])
def test_step_problems_refused(lib, kw, code):
    assert run_step(lib, step(**kw)) == code


def test_step_pointers(lib):
    for k in ("x", "dt", "A", "B", "C", "states", "out"):
        assert run_step(lib, step(), null=(k,)) == BAD
    for k in ("x", "dt", "B", "C", "states", "out"):
        assert run_step(lib, step(), odd=(k,)) == BAD
    assert lib.ssd_step(None, *[FAKE] * 10, None) == BAD
    everything = ("x", "dt", "bias", "A", "B", "C", "D", "states", "out")
    assert run_step(lib, step(batch=0, nslots=0), null=everything) == b.SSD_OK


def norm(**kw):
    base = dict(tokens=10, channels=96, dtype=b.SSD_BF16, residual_dtype=b.SSD_F32,
                gate_activation=1, residual_scale=1.0, eps=1e-5)
    base.update(kw)
    return b.BlockNormProblemC(**base)


def norm_fwd(lib, p, x=FAKE, res=FAKE, gate=None, pre=FAKE, out=FAKE, rout=FAKE):
    return lib.ssd_block_norm_fwd(ctypes.byref(p), x, res, gate, None, None, pre, out, rout, None)


def norm_bwd(lib, p, x=FAKE, gate=None, post=None, scale=None, dout=FAKE, dx=FAKE, dgate=None,
             dpost=None, dscale=None, dpre=FAKE, ws=FAKE, size=1 << 40):
    return lib.ssd_block_norm_bwd(ctypes.byref(p), x, FAKE, gate, post, scale, FAKE, dout, None, dx,
                                  None, dgate, dpost, dscale, dpre, ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), BAD), (dict(channels=0), BAD), (dict(dtype=2), BAD),
    (dict(residual_dtype=2), BAD), (dict(dtype=b.SSD_F32, residual_dtype=b.SSD_BF16), BAD),
    (dict(gate_activation=3), BAD), (dict(gate_activation=-1), BAD), (dict(eps=-1e-5), BAD),
    (dict(eps=NAN), BAD), (dict(eps=INF), BAD), (dict(residual_scale=NAN), BAD),
    (dict(residual_scale=INF), BAD), (dict(channels=8193), UNS), (dict(tokens=1 << 41), UNS),
    (dict(tokens=1 << 62), UNS), (dict(tokens=1 << 38), UNS),
])
def test_block_norm_problems_refused(lib, kw, code):
    p = norm(**kw)
    assert norm_fwd(lib, p) == norm_bwd(lib, p) == code
    assert lib.ssd_block_norm_bwd_workspace_size(ctypes.byref(p)) == 0


def test_block_norm_pointers(lib):
    p = norm()
    for kw in (dict(x=None), dict(pre=None), dict(out=None), dict(x=ODD), dict(res=ODD),
               dict(gate=ODD), dict(out=ODD), dict(rout=ODD)):
        assert norm_fwd(lib, p, **kw) == BAD, kw
    for kw in (dict(x=None), dict(dout=None), dict(dx=None), dict(dpre=None), dict(gate=FAKE),
               dict(dgate=FAKE), dict(post=FAKE), dict(dpost=FAKE), dict(scale=FAKE),
               dict(dscale=FAKE), dict(dout=ODD)):
        assert norm_bwd(lib, p, **kw) == BAD, kw
    need = lib.ssd_block_norm_bwd_workspace_size(ctypes.byref(p))
    assert need > 0 and need % 256 == 0
    assert norm_bwd(lib, p, ws=None) == WSP
    assert norm_bwd(lib, p, size=need - 1) == WSP
    assert norm_bwd(lib, p, ws=ctypes.c_void_p(0x1010)) == WSP
    empty = norm(tokens=0)
    assert lib.ssd_block_norm_fwd(ctypes.byref(empty), *[None] * 8, None) == b.SSD_OK


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    w, v = torch.zeros(8, 4), torch.zeros(8)
    for call in (lambda: b.conv_fwd(x, w), lambda: b.conv_bwd(x, w, [x]),
                 lambda: b.conv_step(x[0], torch.zeros(4, 3, 8), w),
                 lambda: b.ssd_step(x, x[..., 0], v, x, x, torch.zeros(1, 4, 8, 8)),
                 lambda: b.block_norm_fwd(x, x, v), lambda: b.block_norm_bwd(x, x, v, x)):
        with pytest.raises(ValueError, match="GPU only"):
            call()


def test_row_strides_of_the_binding():
    """Rows inside wider rows are taken, anything a kernel could not address is
    refused."""
    wide = torch.zeros(2, 5, 40)
    f = b._row_stride
    assert f(wide[..., 8:24], "x", 2) == 40
    assert f(wide[..., :16].contiguous(), "x", 2) == 16
    assert f(wide[:, 0, 8:24], "x", 1) == 200
    assert f(wide[:1, :1, 8:24], "x", 2) == 16               # one row: no distance
    assert f(wide[:, :1, 8:24], "x", 2) == 200
    assert f(wide[0, :, :24].unflatten(1, (3, 8)), "x", 1) == 40
    assert f(wide[:, :0], "x", 2) == 40
    for t, rows in ((wide.transpose(1, 2), 2),               # channels not contiguous
                    (wide[..., ::2], 2),
                    (wide[:, :3, :16], 2),                   # batch rows further apart
                    (wide[0, 0].expand(4, 40), 1),           # overlapping rows
                    (wide[0, :, :24].unflatten(1, (3, 8))[..., :4], 1)):
        with pytest.raises(ValueError):
            f(t, "x", rows)
