"""The single-token state update on the GPU against the fp64 oracle.  Every
element is held to the count of operations (tests/layer_bounds.py):
  delta  u = dt + bias rounds once, |u| U relative to softplus (its slope never
         exceeds its value); exp, log1p and the sum add 12 U:  (12 + |u|) U
  decay  |delta A| (err(delta) + U) + 6 U relative
  state  |decay h| (err(decay) + 2 U) + |delta x B| (err(delta) + 4 U)
  y      sum |C| err(state), and 24 U of the sum of |h C| (at most 4 values a
         lane, 6 exchanges, the products) + 3 U |D x|
"""
import math

import numpy as np
import pytest
import torch

from oracle import layer
from oracle.recurrence import to_f64
from state_space_model_ssd_amd import binding
from tests.layer_bounds import DT, RND, TINY, U, check

pytestmark = pytest.mark.gpu

CASES = {
    # (batch, nslots, H, P, N, G, dtype, dt dtype, pad, slots, bias, D, clamp)
    "layer": (2, 2, 24, 64, 128, 1, "bf16", "bf16", 100, None, True, True, None),
    "one": (1, 1, 1, 1, 1, 1, "f32", "f32", 0, None, True, True, None),
    "groups": (5, 8, 8, 64, 128, 4, "bf16", "f32", 0, [7, 0, 3, 1, 2], True, True, None),
    "padding": (7, 4, 4, 32, 16, 2, "bf16", "bf16", 3, [2, -1, 2, 3, 0, 99, -2 ** 31], True, True, None),
    "small-f32": (3, 3, 4, 32, 16, 1, "f32", "f32", 5, None, False, False, None),
    "n256": (2, 3, 2, 64, 256, 1, "bf16", "bf16", 0, [2, 1], True, True, None),
    "n255": (2, 3, 2, 50, 255, 1, "bf16", "f32", 1, [0, 2], True, False, None),
    "n130": (2, 2, 2, 5, 130, 2, "f32", "f32", 0, None, False, True, None),
    "n100-odd-p": (3, 3, 6, 33, 100, 3, "bf16", "bf16", 7, None, True, True, None),
    "n65": (2, 2, 1, 17, 65, 1, "f32", "f32", 0, None, True, True, None),
    "n33": (2, 2, 3, 9, 33, 1, "bf16", "bf16", 0, None, True, True, None),
    "n7": (2, 2, 3, 100, 7, 3, "f32", "f32", 0, None, True, True, None),
    "n4": (2, 2, 2, 130, 4, 1, "bf16", "bf16", 0, None, True, True, None),
    "wide-head": (1, 1, 2, 300, 48, 1, "bf16", "bf16", 0, None, True, True, None),
    "clamped": (3, 3, 4, 64, 128, 1, "bf16", "bf16", 0, None, True, True, (0.05, 0.2)),
    "many-rows": (600, 610, 2, 8, 16, 1, "bf16", "bf16", 0, "shuffle", True, True, None),
}


def draw(name):
    batch, nslots, H, P, N, G, dtype, dtd, pad, slots, bias, D, clamp = CASES[name]
    g = torch.Generator().manual_seed(len(name) + N)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    row = r(batch, H * P + 2 * G * N + pad).to(DT[dtype])
    d = dict(row=row, x=row[:, :H * P].unflatten(1, (H, P)),
             B=row[:, H * P:H * P + G * N].unflatten(1, (G, N)),
             C=row[:, H * P + G * N:H * P + 2 * G * N].unflatten(1, (G, N)),
             dt=(r(batch, H) * 2 - 1).to(DT[dtd]), A=-torch.exp(r(H)), D=r(H) if D else None,
             bias=r(H) if bias else None, states=r(nslots, H, P, N))
    if slots == "shuffle":
        slots = torch.randperm(nslots, generator=g)[:batch].tolist()
        slots[7], slots[333], slots[599] = -1, slots[3], slots[598]
    kw = {} if clamp is None else dict(dt_min=clamp[0], dt_max=clamp[1])
    return d, slots, kw


def device(d):
    e = {k: None if v is None else v.cuda() for k, v in d.items()}
    H, P = d["x"].shape[1:]
    G, N = d["B"].shape[1:]
    row = e["row"]
    e["x"] = row[:, :H * P].unflatten(1, (H, P))
    e["B"] = row[:, H * P:H * P + G * N].unflatten(1, (G, N))
    e["C"] = row[:, H * P + G * N:H * P + 2 * G * N].unflatten(1, (G, N))
    return e


def bounds(d, slots, dt_min=0.0, dt_max=math.inf):
    """(state, y) error bounds per row (rows as given, padding included)."""
    x, dt, A, B, C, D, bias, states = (to_f64(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias",
                                                              "states"))
    batch, H = dt.shape
    rep = H // B.shape[1]
    B, C = np.repeat(B, rep, 1), np.repeat(C, rep, 1)
    idx = np.arange(batch) if slots is None else np.clip(np.asarray(slots), 0, len(states) - 1)
    u = dt + (bias if bias is not None else 0.0)
    delta = np.clip(np.logaddexp(0, u), dt_min, dt_max)
    de = (12 + np.abs(u)) * U
    decay = np.exp(delta * A)
    ce = np.abs(delta * A) * (de + U) + 6 * U
    h0 = np.abs(decay[..., None, None] * states[idx])
    add = np.abs(delta[..., None, None] * x[..., None] * B[:, :, None, :])
    se = h0 * (ce + 2 * U)[..., None, None] + add * (de + 4 * U)[..., None, None] + TINY
    ye = (np.abs(C)[:, :, None, :] * (se + 24 * U * (h0 + add))).sum(-1)
    if D is not None:
        ye = ye + 3 * U * np.abs(D[:, None] * x)
    return se, ye, idx


@pytest.mark.parametrize("name", sorted(CASES))
def test_step(name):
    dtype = CASES[name][6]
    d, slots, kw = draw(name)
    e = device(d)
    batch, H, P = d["x"].shape
    nslots = d["states"].shape[0]
    out = torch.full((batch, H, P), 5.0, dtype=DT[dtype], device="cuda")
    ds = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    binding.ssd_step(e["x"], e["dt"], e["A"], e["B"], e["C"], e["states"], D=e["D"],
                     dt_bias=e["bias"], slots=ds, out=out, **kw)
    torch.cuda.synchronize()
    ref, sref = layer.ssd_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["states"], d["D"], d["bias"],
                               slots, **kw)
    se, ye, idx = bounds(d, slots, **kw)
    pads = np.array(layer.padding_rows(slots, batch, nslots))
    st = np.zeros_like(sref)                       # states no row has are not touched: bound 0
    st[idx[~pads]] = se[~pads]
    check(e["states"], sref, st, "state")
    assert (out.cpu()[torch.from_numpy(pads)] == 5).all()
    check(out, ref, ye + RND[dtype] * (np.abs(np.nan_to_num(ref)) + ye) + TINY, "out")


def test_step_padding_never_reads_or_writes_values():
    """A padding row of NaN changes nothing; a state of NaN stays in its slot."""
    d, _, _ = draw("groups")
    e = device(d)
    st = e["states"].clone()
    st[5] = float("nan")
    slots = torch.tensor([7, -1, 3, 3, 2], dtype=torch.int32, device="cuda")
    e["row"][1] = float("nan")
    e["row"][3] = float("inf")
    out = binding.ssd_step(e["x"], e["dt"], e["A"], e["B"], e["C"], st, D=e["D"], slots=slots)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and not out[1].any() and not out[3].any()
    assert torch.isfinite(st[[0, 1, 2, 3, 4, 6, 7]]).all() and torch.isnan(st[5]).all()
    for s in (0, 1, 4, 6):
        assert torch.equal(st[s], e["states"][s])


def test_step_no_rows_and_no_slots():
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    st = z(3, 2, 4, 8) + 1
    out = binding.ssd_step(z(0, 2, 4), z(0, 2), z(2), z(0, 1, 8), z(0, 1, 8), st)
    assert out.shape == (0, 2, 4)
    none = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = binding.ssd_step(z(2, 2, 4), z(2, 2), z(2), z(2, 1, 8), z(2, 1, 8), z(0, 2, 4, 8), slots=none)
    torch.cuda.synchronize()
    assert not out.any() and (st == 1).all()


def test_step_far_slots_of_a_long_cache():
    """Slots whose state begins past 2^31 and 2^32 elements of the cache."""
    H, P, N = 32, 64, 128
    per = H * P * N
    nslots = 2 ** 32 // per + 3                    # 17 GB of fp32
    st = torch.empty((nslots, H, P, N), device="cuda")
    slots = [nslots - 1, 2 ** 31 // per, 0, 2 ** 32 // per]
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    d = dict(x=r(4, H, P), dt=r(4, H), A=-torch.exp(r(H)), B=r(4, 1, N), C=r(4, 1, N), D=None, bias=None,
             states=r(4, H, P, N))
    st[slots] = d["states"].cuda()
    out = binding.ssd_step(*(d[k].cuda() for k in ("x", "dt", "A", "B", "C")), st,
                           slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    ref, sref = layer.ssd_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["states"])
    se, ye, _ = bounds(d, None)
    check(st[slots], sref, se, "state")
    check(out, ref, ye + U * np.abs(ref) + TINY, "out")


def test_step_argument_checks():
    d, _, _ = draw("groups")
    e = device(d)
    args = dict(x=e["x"], dt=e["dt"], A=e["A"], B=e["B"], C=e["C"], states=e["states"])
    slots = torch.zeros(5, dtype=torch.int32, device="cuda")
    for bad in (dict(dt=e["dt"].half()), dict(B=e["B"].float()), dict(states=e["states"].bfloat16()),
                dict(states=e["states"][..., ::2]), dict(slots=slots.long()), dict(slots=slots[:4]),
                dict(x=e["x"].transpose(1, 2)), dict(C=e["C"][:3]), dict(D=e["A"].cpu()),
                dict(out=e["x"].float()), dict(dt=e["dt"][:4])):
        with pytest.raises(ValueError):
            binding.ssd_step(**{**dict(slots=slots), **args, **bad})
    with pytest.raises(binding.SsdError) as err:
        binding.ssd_step(**{**args, "states": e["states"][:4]})     # fewer states than rows, no slots
    assert err.value.code == binding.SSD_ERR_INVALID_ARG
    big = torch.zeros((8, 8, 64, 300), device="cuda")
    B = torch.zeros((5, 4, 300), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.SsdError) as err:
        binding.ssd_step(**{**args, "states": big, "B": B, "C": B})
    assert err.value.code == binding.SSD_ERR_UNSUPPORTED
