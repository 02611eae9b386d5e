"""Host-side checks of the gated delta rule and the query/key norm (CPU only: every call
fails, or has nothing to launch, before anything reaches a device)."""
import ctypes

import pytest
import torch

from state_space_model_ssd_amd import binding as b

FAKE = ctypes.c_void_p(0x10000)
BAD, UNS, WSP = b.SSD_ERR_INVALID_ARG, b.SSD_ERR_UNSUPPORTED, b.SSD_ERR_WORKSPACE
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return b.load_library()


# pointers far apart, so that none of the calls is refused for shared memory
def at(i):
    return ctypes.c_void_p((i + 1) << 44)


def delta(**kw):
    base = dict(batch=2, seqlen=100, nheads=8, headdim=64, dstate=128, ngroups=4, nseq=0,
                dtype=b.SSD_BF16, gate_dtype=b.SSD_F32, scale=0.1, clear_outside=0)
    base.update(kw)
    return b.DeltaProblemC(**base)


FWD = ("q", "k", "v", "g", "beta", "init", "cu", "out", "final", "ws")
BWD = ("q", "k", "v", "g", "beta", "init", "cu", "dout", "dfinal", "dq", "dk", "dv", "dg", "dbeta",
       "dinit", "ws")


def call(lib, fn, names, p, size=1 << 43, **given):
    ptr = {n: at(i) for i, n in enumerate(names)}
    ptr["cu"] = None
    ptr.update(given)
    return getattr(lib, fn)(ctypes.byref(p), *[ptr[n] for n in names], size, None)


def fwd(lib, p, **kw):
    return call(lib, "ssd_delta_fwd", FWD, p, **kw)


def bwd(lib, p, **kw):
    return call(lib, "ssd_delta_bwd", BWD, p, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(seqlen=-1), BAD), (dict(nseq=-1), BAD), (dict(nheads=0), BAD),
    (dict(headdim=0), BAD), (dict(dstate=0), BAD), (dict(ngroups=0), BAD), (dict(ngroups=3), BAD),
    (dict(dtype=2), BAD), (dict(gate_dtype=-1), BAD), (dict(dtype=b.SSD_F32, gate_dtype=b.SSD_BF16), BAD),
    (dict(scale=NAN), BAD), (dict(scale=INF), BAD), (dict(clear_outside=2), BAD), (dict(nseq=3), BAD),
    (dict(dstate=96), UNS), (dict(dstate=256), UNS), (dict(headdim=72), UNS), (dict(headdim=272), UNS),
    (dict(nheads=8192), UNS), (dict(batch=65536), UNS), (dict(seqlen=2 ** 30 + 1), UNS),
    (dict(batch=1024, seqlen=2 ** 20 + 1), UNS), (dict(batch=1, nseq=65536), UNS),
    (dict(batch=1, seqlen=2 ** 25 + 1), UNS), (dict(batch=1025, nheads=4096, seqlen=1, headdim=16), UNS),
    (dict(batch=129, nheads=4096, headdim=256, seqlen=0), UNS),
])
def test_delta_problems_refused(lib, kw, code):
    p = delta(**kw)
    assert fwd(lib, p) == bwd(lib, p) == code
    assert lib.ssd_delta_fwd_workspace_size(ctypes.byref(p)) == 0
    assert lib.ssd_delta_bwd_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("kw", [
    dict(dstate=32, headdim=16), dict(headdim=256, nheads=4096, ngroups=4096, batch=1),
    dict(batch=65535, seqlen=1), dict(batch=1, nseq=65535), dict(batch=1, seqlen=2 ** 25),
    dict(batch=1, seqlen=2 ** 28, nheads=1, ngroups=1), dict(batch=1024, nheads=4096, seqlen=1, headdim=32),
])
def test_delta_limits_taken(lib, kw):
    p = delta(**kw)
    need = lib.ssd_delta_fwd_workspace_size(ctypes.byref(p))
    assert need > 0 and need % 256 == 0
    assert lib.ssd_delta_bwd_workspace_size(ctypes.byref(p)) > need
    assert fwd(lib, p, q=None) == BAD                       # a size that is taken, no input


def test_delta_workspace(lib):
    for fn, run in ((lib.ssd_delta_fwd_workspace_size, fwd), (lib.ssd_delta_bwd_workspace_size, bwd)):
        p = delta()
        need = fn(ctypes.byref(p))
        assert run(lib, p, ws=None) == run(lib, p, size=need - 1) == WSP
        assert run(lib, p, ws=ctypes.c_void_p((99 << 44) + 8)) == WSP
        # pairs are kept, in twice the room, where the gates' gradients are fp32 or few
        big = dict(batch=4, seqlen=8192)
        if run is bwd:
            assert fn(ctypes.byref(delta(**big))) > fn(ctypes.byref(delta(**big, gate_dtype=b.SSD_BF16)))
            few = dict(seqlen=64)
            assert fn(ctypes.byref(delta(**few))) == fn(ctypes.byref(delta(**few, gate_dtype=b.SSD_BF16)))


def test_delta_pointers_and_packing(lib):
    p = delta()
    odd = ctypes.c_void_p((99 << 44) + 8)                   # aligned to 8, not to 16
    for n in ("q", "k", "v", "g", "beta", "out"):
        assert fwd(lib, p, **{n: None}) == BAD, n
    for n in ("q", "k", "v", "out"):
        assert fwd(lib, p, **{n: odd}) == BAD, n
    for n in ("g", "beta", "init", "final"):
        assert fwd(lib, p, **{n: ctypes.c_void_p((99 << 44) + 2)}) == BAD, n
    for n in ("q", "k", "v", "g", "beta", "dout", "dq", "dk", "dv", "dg", "dbeta"):
        assert bwd(lib, p, **{n: None}) == BAD, n
    for n in ("dout", "dq", "dk", "dv"):
        assert bwd(lib, p, **{n: odd}) == BAD, n
    for n in ("dg", "dbeta", "dfinal", "dinit"):
        assert bwd(lib, p, **{n: ctypes.c_void_p((99 << 44) + 2)}) == BAD, n
    assert fwd(lib, p, cu=at(50)) == bwd(lib, p, cu=at(50)) == BAD             # rows take no cu_seqlens
    packed = delta(batch=1, nseq=3)
    assert fwd(lib, packed) == bwd(lib, packed) == BAD                         # a packed batch does
    assert fwd(lib, packed, cu=at(50), ws=None) == WSP
    assert lib.ssd_delta_fwd(None, *[FAKE] * 10, 0, None) == BAD
    assert lib.ssd_delta_bwd(None, *[FAKE] * 16, 0, None) == BAD


def test_delta_shared_memory_is_refused(lib):
    p = delta()
    for w, r in (("out", "v"), ("out", "q"), ("final", "init"), ("ws", "k"), ("final", "out"), ("out", "beta")):
        assert fwd(lib, p, **{w: at(60), r: at(60)}) == BAD, (w, r)
    for w, r in (("dv", "dout"), ("dq", "q"), ("dk", "dq"), ("dinit", "dfinal"), ("dg", "beta"),
                 ("dbeta", "dg"), ("ws", "dout"), ("dv", "v")):
        assert bwd(lib, p, **{w: at(60), r: at(60)}) == BAD, (w, r)


def test_delta_nothing_to_do(lib):
    """No sequences: ok without a launch, whatever else is missing but the workspace."""
    p = delta(batch=0)
    assert fwd(lib, p, **{n: None for n in FWD if n != "ws"}) == b.SSD_OK
    assert bwd(lib, p, **{n: None for n in BWD if n != "ws"}) == b.SSD_OK


def step(**kw):
    base = dict(batch=2, nheads=8, headdim=64, dstate=128, ngroups=2, nslots=4, q_stride=0, k_stride=0,
                v_stride=0, g_stride=0, beta_stride=0, dtype=b.SSD_BF16, gate_dtype=b.SSD_F32, scale=1.0)
    base.update(kw)
    return b.DeltaStepProblemC(**base)


STEP = ("q", "k", "v", "g", "beta", "states", "slots", "out")


def run_step(lib, p, **given):
    ptr = {n: at(i) for i, n in enumerate(STEP)}
    ptr["slots"] = None
    ptr.update(given)
    return lib.ssd_delta_step(ctypes.byref(p), *[ptr[n] for n in STEP], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(nheads=0), BAD), (dict(headdim=0), BAD), (dict(dstate=0), BAD),
    (dict(ngroups=0), BAD), (dict(ngroups=3), BAD), (dict(nslots=-1), BAD), (dict(nslots=1), BAD),
    (dict(dtype=2), BAD), (dict(gate_dtype=2), BAD), (dict(dtype=b.SSD_F32, gate_dtype=b.SSD_BF16), BAD),
    (dict(scale=NAN), BAD), (dict(q_stride=255), BAD), (dict(k_stride=-1), BAD), (dict(v_stride=511), BAD),
    (dict(g_stride=7), BAD), (dict(beta_stride=1), BAD), (dict(v_stride=2 ** 31 + 1), BAD),
    (dict(dstate=257), UNS), (dict(batch=65536, nslots=65536), UNS), (dict(nheads=65536, ngroups=1), UNS),
    (dict(headdim=65536), UNS), (dict(nslots=2 ** 31), UNS), (dict(batch=65535, nslots=65535, nheads=1024), UNS),
])
def test_step_problems_refused(lib, kw, code):
    assert run_step(lib, step(**kw)) == code


def test_step_pointers(lib):
    for n in ("q", "k", "v", "g", "beta", "states", "out"):
        assert run_step(lib, step(), **{n: None}) == BAD
        assert run_step(lib, step(), **{n: ctypes.c_void_p((99 << 44) + 1)}) == BAD
    for w, r in (("out", "v"), ("states", "out"), ("out", "q"), ("states", "beta")):
        assert run_step(lib, step(), **{w: at(60), r: at(60)}) == BAD
    # queries, keys and values may be columns of one row, the output none of them
    base = at(60).value
    cols = dict(q=ctypes.c_void_p(base), k=ctypes.c_void_p(base + 512), v=ctypes.c_void_p(base + 1024))
    p = step(q_stride=1024, k_stride=1024, v_stride=1024)
    assert run_step(lib, p, **cols, out=ctypes.c_void_p(base + 2048 * 4), states=None) == BAD
    assert run_step(lib, step(batch=0, nslots=0), **{n: None for n in STEP}) == b.SSD_OK
    assert lib.ssd_delta_step(None, *[FAKE] * 8, None) == BAD


def norm(**kw):
    base = dict(tokens=10, q_heads=4, k_heads=2, headdim=64, rotary_pairs=32, q_stride=0, k_stride=0,
                dq_stride=0, dk_stride=0, dtype=b.SSD_BF16, norm=0, interleaved=0, eps=1e-6)
    base.update(kw)
    return b.QkNormProblemC(**base)


NF = ("q", "k", "qw", "kw", "pos", "freq", "qo", "ko")
NB = ("q", "k", "qw", "kw", "pos", "freq", "dqo", "dko", "dq", "dk", "dqw", "dkw", "ws")


def nfwd(lib, p, **given):
    ptr = {n: at(i) for i, n in enumerate(NF)}
    ptr.update(given)
    return lib.ssd_qk_norm_fwd(ctypes.byref(p), *[ptr[n] for n in NF], None)


def nbwd(lib, p, size=1 << 40, **given):
    ptr = {n: at(i) for i, n in enumerate(NB)}
    ptr.update(given)
    return lib.ssd_qk_norm_bwd(ctypes.byref(p), *[ptr[n] for n in NB], size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), BAD), (dict(q_heads=0), BAD), (dict(k_heads=0), BAD), (dict(headdim=0), BAD),
    (dict(rotary_pairs=-1), BAD), (dict(rotary_pairs=33), BAD), (dict(dtype=3), BAD), (dict(norm=2), BAD),
    (dict(interleaved=2), BAD), (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD),
    (dict(q_stride=255), BAD), (dict(k_stride=1), BAD), (dict(dq_stride=-3), BAD), (dict(dk_stride=127), BAD),
    (dict(q_stride=2 ** 31 + 1), BAD),
    (dict(headdim=257), UNS), (dict(q_heads=4097), UNS), (dict(k_heads=4097), UNS), (dict(tokens=2 ** 30 + 1), UNS),
])
def test_norm_problems_refused(lib, kw, code):
    p = norm(**kw)
    assert nfwd(lib, p) == nbwd(lib, p) == code
    assert lib.ssd_qk_norm_bwd_workspace_size(ctypes.byref(p)) == 0


def test_norm_pointers(lib):
    odd = ctypes.c_void_p((99 << 44) + 1)
    p = norm()
    for n in ("q", "k", "pos", "freq", "qo", "ko"):
        assert nfwd(lib, p, **{n: None}) == BAD, n
        assert nfwd(lib, p, **{n: odd}) == BAD, n
    for n in ("q", "k", "pos", "freq", "dqo", "dko", "dq", "dk"):
        assert nbwd(lib, p, **{n: None}) == BAD, n
    # a weight has a gradient, and only a weight
    for n in ("qw", "kw", "dqw", "dkw"):
        assert nbwd(lib, p, **{n: None}) == BAD, n
    need = lib.ssd_qk_norm_bwd_workspace_size(ctypes.byref(p))
    assert need > 0 and need % 256 == 0
    assert nbwd(lib, p, ws=None) == nbwd(lib, p, size=need - 1) == WSP
    assert nbwd(lib, p, ws=ctypes.c_void_p((99 << 44) + 8)) == WSP
    for w, r in (("qo", "q"), ("ko", "q"), ("ko", "qo"), ("qo", "kw"), ("ko", "pos")):
        assert nfwd(lib, p, **{w: at(60), r: at(60)}) == BAD, (w, r)
    for w, r in (("dq", "dqo"), ("dk", "k"), ("dqw", "qw"), ("dkw", "dqw"), ("ws", "dk"), ("dq", "freq")):
        assert nbwd(lib, p, **{w: at(60), r: at(60)}) == BAD, (w, r)
    assert lib.ssd_qk_norm_fwd(None, *[FAKE] * 8, None) == BAD
    assert lib.ssd_qk_norm_bwd(None, *[FAKE] * 13, 0, None) == BAD
    empty = norm(tokens=0)
    assert nfwd(lib, empty, **{n: None for n in NF}) == b.SSD_OK


def test_binding_refuses_on_the_host():
    z = torch.zeros
    cases = [
        lambda: b.delta_fwd(z(1, 4, 2, 32), z(1, 4, 2, 32), z(1, 4, 4, 16), z(1, 4, 4), z(1, 4, 4)),
        lambda: b.delta_step(z(1, 2, 32), z(1, 2, 32), z(1, 4, 16), z(1, 4), z(1, 4), z(1, 4, 16, 32)),
        lambda: b.qk_norm_fwd(z(4, 2, 32), z(4, 2, 32)),
        lambda: b.qk_norm_bwd(z(4, 2, 32), z(4, 2, 32), z(4, 2, 32), z(4, 2, 32)),
    ]
    for c in cases:
        with pytest.raises(ValueError, match="GPU only"):
            c()
