"""The norms around a block on the GPU, forward and backward, against the fp64
oracle.  Every element is held to a count of operations (tests/layer_bounds.py).
A sum of squares or of a row's products passes at most 2 x 8 values of a lane,
6 exchanges and 16 waves, 38 additions, and its mean one product: 40 U of the sum
of absolute values.  So r1 is off by 20 U + 2 U + U relative (half of the sum's,
the root, eps' sum): 24 U.
  p    x r1 post_w: 26 U relative;  u: + the sigmoid's and 2 U (a bound for all
       three acts: E = 28 U + 2 sigmoid_err + U)
  h    |f u| (E + 2 U) + U |h|;  r2 as r1, and h's own error by its norm
  out  |out| (err(r2) + 2 U) + r2 |pre_w| err(h)
Backward, with T1 = r2 (|dn| + |n| mean|dn n|) + |dh_out| the size of dh's terms:
  n    N = err(r2) + err(h) / |h| enters dn n and n once each and the mean once,
       4 N + 60 U of T1 in all
  du, dp, dgate, dx multiply by p, act, act' (2 E + 40 U covers each) and dx
  repeats the mean over a row: errors of the row's dm by its norms
  weights' gradients: the terms' own errors, + 100 U of their absolute sums (rows
       one after another, at most 40 in these shapes, 4 + 16 + 32 partial sums)
"""
import numpy as np
import pytest
import torch

from oracle import layer
from oracle.recurrence import to_f64
from state_space_model_ssd_amd import binding
from tests.layer_bounds import DT, RND, TINY, U, check, sigmoid_err

pytestmark = pytest.mark.gpu

CASES = {
    # (tokens, channels, dtype, residual dtype, gate, post, scale, alpha, residual given)
    "decode": (4, 768, "bf16", "f32", None, False, False, 1.0, True),
    "all": (130, 2048, "bf16", "bf16", "silu", True, True, 0.22, True),
    "sigmoid": (77, 768, "bf16", "f32", "sigmoid", True, True, 1.0, True),
    "linear": (33, 512, "f32", "f32", "linear", True, False, 0.5, True),
    "first-block": (19, 1536, "bf16", "f32", None, True, True, 1.0, False),
    "scale-only": (9, 1024, "bf16", "bf16", None, False, True, -0.7, True),
    "gate-only": (65, 256, "f32", "f32", "silu", False, False, 1.0, True),
    "odd-f32": (101, 1025, "f32", "f32", None, False, False, 0.5, True),
    "odd-bf16": (50, 771, "bf16", "f32", "sigmoid", True, True, 1.0, True),
    "odd-wide": (12, 4099, "bf16", "bf16", "silu", True, True, 1.0, True),
    "widest-bf16": (5, 8192, "bf16", "f32", "silu", True, True, 1.0, True),
    "widest-f32": (5, 8192, "f32", "f32", "silu", True, True, 1.0, True),
    "wide-odd-f32": (3, 8191, "f32", "f32", None, True, False, 1.0, True),
    "one-channel": (7, 1, "bf16", "bf16", "linear", True, True, 1.0, True),
    "three-channels": (300, 3, "f32", "f32", "silu", True, True, 1.0, True),
    "one-row": (1, 2056, "bf16", "f32", None, True, False, 1.0, True),
    "no-scale": (3000, 64, "bf16", "f32", "sigmoid", False, False, 0.0, True),
    "many-rows": (9000, 40, "f32", "f32", "linear", True, True, 1.0, True),
}


def draw(name):
    T, C, dtype, rdt, gate, post, scale, alpha, res = CASES[name]
    g = torch.Generator().manual_seed(T + C)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    d = dict(x=r(T, C).to(DT[dtype]), residual=(3 * r(T, C)).to(DT[rdt]) if res else None,
             pre=1 + 0.3 * r(C), gate=(2 * r(T, C)).to(DT[dtype]) if gate else None,
             post=1 + 0.3 * r(C) if post else None, scale=1 + 0.3 * r(C) if scale else None,
             dout=r(T, C).to(DT[dtype]), dh=r(T, C).to(DT[rdt]))
    return d, dict(kind=gate or "linear", alpha=alpha, eps=1e-5), dtype, rdt


def device(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def call(d, kw):
    return dict(gate=d["gate"], gate_activation=kw["kind"], post_weight=d["post"], scale=d["scale"],
                residual_scale=kw["alpha"], eps=kw["eps"])


def parts(d, kw):
    """The fp64 quantities of the bounds above."""
    x, res, pre, gate, post, scale = (to_f64(d[k]) for k in ("x", "residual", "pre", "gate", "post", "scale"))
    a = kw["alpha"]
    o = dict(x=x, pre=pre, f=a * (scale if scale is not None else np.ones_like(pre)), post=post, a=a)
    o["r1"] = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + kw["eps"]) if post is not None else 1.0
    o["m"] = x * o["r1"]
    o["p"] = o["m"] * post if post is not None else x
    o["act"], o["dact"] = layer.gate_act(kw["kind"], gate) if gate is not None else (np.ones_like(x), np.zeros_like(x))
    o["E"] = 28 * U + (2 * sigmoid_err(gate) + U if gate is not None else 0.0)
    u = o["p"] * o["act"]
    h = o["f"] * u + (res if res is not None else 0.0)
    o["u"], o["h"] = u, h
    o["eh"] = np.abs(o["f"] * u) * (o["E"] + 2 * U) + U * np.abs(h) + TINY
    o["r2"] = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + kw["eps"])
    norm = np.sqrt((h * h).mean(1, keepdims=True)) + np.sqrt(kw["eps"])
    o["e2"] = 24 * U + np.sqrt((o["eh"] ** 2).mean(1, keepdims=True)) / norm
    return o


@pytest.mark.parametrize("name", sorted(CASES))
def test_block_norm_forward(name):
    d, kw, dtype, rdt = draw(name)
    e = device(d)
    out, h = binding.block_norm_fwd(e["x"], e["residual"], e["pre"], residual_dtype=DT[rdt], **call(e, kw))
    torch.cuda.synchronize()
    ref, href = layer.block_norm_fwd(d["x"], d["residual"], d["pre"], d["gate"], kw["kind"], d["post"],
                                     d["scale"], kw["alpha"], kw["eps"])
    o = parts(d, kw)
    check(h, href, o["eh"] + RND[rdt] * (np.abs(href) + o["eh"]), "residual_out")
    tol = np.abs(ref) * (o["e2"] + 2 * U) + o["r2"] * np.abs(o["pre"]) * o["eh"]
    check(out, ref, tol + RND[dtype] * (np.abs(ref) + tol), "out")


def row_mean(v):
    return v.mean(1, keepdims=True)


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("with_dh", [True, False])
def test_block_norm_backward(name, with_dh):
    d, kw, dtype, rdt = draw(name)
    if not with_dh:
        d["dh"] = None
    e = device(d)
    g = binding.block_norm_bwd(e["x"], e["residual"], e["pre"], e["dout"], e["dh"], residual_dtype=DT[rdt],
                               **call(e, kw))
    torch.cuda.synchronize()
    r = layer.block_norm_bwd(d["x"], d["residual"], d["pre"], d["dout"], d["dh"], d["gate"], kw["kind"],
                             d["post"], d["scale"], kw["alpha"], kw["eps"])
    o = parts(d, kw)
    ab = np.abs
    do = ab(to_f64(d["dout"]))
    n, en = ab(o["h"]) * o["r2"], o["r2"] * o["eh"] + ab(o["h"]) * o["r2"] * (o["e2"] + U)
    dn = do * ab(o["pre"])
    # errors of n in the terms themselves, the relative ones of r2 and the sums
    e_dh = o["r2"] * (dn * (o["e2"] + 4 * U) + en * row_mean(dn * n) + n * row_mean(dn * en)
                      + n * row_mean(dn * n) * (2 * o["e2"] + 60 * U)) + TINY
    dh = ab(r["residual"])
    e_dh = e_dh + 4 * U * (o["r2"] * (dn + n * row_mean(dn * n)) + dh)
    f, p, act, dact, m = ab(o["f"]), ab(o["p"]), ab(o["act"]), ab(o["dact"]), ab(o["m"])
    E = 2 * o["E"] + 40 * U
    tols = {"residual": e_dh, "pre_weight": (do * en).sum(0) + 100 * U * (do * n).sum(0)}
    if d["scale"] is not None:
        s = ab(o["a"]) * p * act
        tols["scale"] = (s * (e_dh + E * dh)).sum(0) + 100 * U * (s * dh).sum(0)
    if d["gate"] is not None:
        # act' is a difference of terms of size up to 1 + |z|
        z = ab(to_f64(d["gate"])) if kw["kind"] == "silu" else 0.0
        size = dact + (sigmoid_size(d["gate"]) * (1 + z) if kw["kind"] != "linear" else 0.0)
        tols["gate"] = f * p * (dact * (e_dh + E * dh) + size * E * dh)
    e_dp = f * act * (e_dh + E * dh)
    dp = f * act * dh
    if d["post"] is not None:
        w = ab(o["post"])
        tols["post_weight"] = (m * (e_dp + 26 * U * dp)).sum(0) + 100 * U * (m * dp).sum(0)
        dm, e_dm = dp * w, e_dp * w + 2 * U * dp * w
        tols["x"] = o["r1"] * (e_dm + 30 * U * dm + m * row_mean(m * e_dm) + 120 * U * m * row_mean(m * dm))
    else:
        tols["x"] = e_dp
    given = {"residual": "residual", "gate": "gate", "post_weight": "post", "scale": "scale"}
    for k in ("x", "residual", "gate", "post_weight", "scale", "pre_weight"):
        if k in given and d[given[k]] is None:
            assert g[k] is None
            continue
        rnd = RND[rdt] if k == "residual" else RND[dtype] if k in ("x", "gate") else U
        tol = tols[k] + TINY
        check(g[k], r[k], tol + rnd * (ab(r[k]) + tol), "d" + k)


def sigmoid_size(gate):
    return 1.0 / (1.0 + np.exp(-to_f64(gate)))


def test_block_norm_in_place_and_deterministic():
    d, kw, dtype, rdt = draw("all")
    e = device(d)
    out, h = binding.block_norm_fwd(e["x"], e["residual"], e["pre"], **call(e, kw))
    x, res = e["x"].clone(), e["residual"].clone()
    binding.block_norm_fwd(x, res, e["pre"], out=x, residual_out=res, **call(e, kw))
    g, k = (binding.block_norm_bwd(e["x"], e["residual"], e["pre"], e["dout"], e["dh"], **call(e, kw))
            for _ in range(2))
    torch.cuda.synchronize()
    assert torch.equal(x, out) and torch.equal(res, h)
    for n in g:
        if n != "workspace":
            assert torch.equal(g[n], k[n])


@pytest.mark.parametrize("C", [64, 300, 2048, 5000])
def test_block_norm_in_place_over_many_rows(C):
    """In place where a workgroup walks over several rows with the next row's
    loads in flight."""
    g = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn((6001, C), generator=g, device="cuda", dtype=torch.bfloat16)
    res, w = torch.randn((6001, C), generator=g, device="cuda"), torch.rand(C, generator=g, device="cuda")
    kw = dict(post_weight=w, scale=w, residual_scale=0.5)
    out, h = binding.block_norm_fwd(x, res, w, **kw)
    binding.block_norm_fwd(x, res, w, out=x, residual_out=res, **kw)
    torch.cuda.synchronize()
    assert torch.equal(x, out) and torch.equal(res, h)


def test_block_norm_far_rows():
    """Elements past 2^32: the last rows equal a run on those rows alone."""
    C = 8192
    T = 2 ** 32 // C + 3000
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.full((T, C), 0.25, dtype=torch.bfloat16, device="cuda")
    x[-2000:] = torch.randn((2000, C), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(C, generator=g, device="cuda")
    out, h = binding.block_norm_fwd(x, x, w, post_weight=w)
    o2, h2 = binding.block_norm_fwd(x[-2000:], x[-2000:], w, post_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(out[-2000:], o2) and torch.equal(h[-2000:], h2)
    del out
    gr = binding.block_norm_bwd(x, x, w, h, post_weight=w)
    wg = binding.block_norm_bwd(x[-2000:], x[-2000:], w, h[-2000:], post_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(gr["x"][-2000:], wg["x"]) and torch.equal(gr["residual"][-2000:], wg["residual"])


def test_block_norm_rows_are_independent():
    """Infinity, NaN and zeros in some rows leave the others as they were."""
    d, kw, dtype, rdt = draw("sigmoid")
    e = device(d)
    out, h = binding.block_norm_fwd(e["x"], e["residual"], e["pre"], **call(e, kw))
    g = binding.block_norm_bwd(e["x"], e["residual"], e["pre"], e["dout"], e["dh"], **call(e, kw))
    x, res = e["x"].clone(), e["residual"].clone()
    x[3], x[40, 5], res[9, 0], x[11], res[11] = float("nan"), float("inf"), float("inf"), 0, 0
    o2, h2 = binding.block_norm_fwd(x, res, e["pre"], **call(e, kw))
    g2 = binding.block_norm_bwd(x, res, e["pre"], e["dout"], e["dh"], **call(e, kw))
    torch.cuda.synchronize()
    keep = [i for i in range(77) if i not in (3, 40, 9, 11)]
    assert torch.equal(out[keep], o2[keep]) and torch.equal(h[keep], h2[keep])
    for k in ("x", "residual", "gate"):
        assert torch.equal(g[k][keep], g2[k][keep])
    assert not o2[11].any() and torch.isfinite(g2["x"][11]).all()    # a row of zeros: eps holds


@pytest.mark.parametrize("C", [700, 701, 2300])
def test_block_norm_infinite_values_as_the_formula(C):
    """Rows that do not fill their waves: infinity at one channel reaches the
    others exactly as the formula says (here h's sum is infinite, so every other
    output is zero)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, res, gate, w = r(8, C), r(8, C), r(8, C).abs() + 0.1, torch.ones(C, device="cuda")
    for row, t in ((0, x), (1, res), (2, gate)):
        t[row, 0] = float("inf")
    x[3, C - 1] = float("inf")
    for post in (None, w):
        out, h = binding.block_norm_fwd(x, res, w, gate=gate, gate_activation="linear", post_weight=post)
        xs = x if post is None else x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5)
        hr = res + xs * gate
        ref = hr * torch.rsqrt((hr * hr).mean(1, keepdim=True) + 1e-5)
        torch.cuda.synchronize()
        for got, want in ((out, ref), (h, hr)):
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(torch.isinf(got), torch.isinf(want))
            fin = torch.isfinite(want)
            assert torch.allclose(got[fin], want[fin], rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("k", [46, -46])
@pytest.mark.parametrize("C,post", [(768, True), (768, False), (1025, True), (4096, True)])
def test_block_norm_backward_holds_at_any_scale_of_the_stream(C, post, k):
    """Without eps, a stream 2^k times as large gives the same out and the same
    gradients, dresidual 2^-k times as large: products with powers of two are
    exact.  Only the root of the mean may round otherwise, by 2 U on either side,
    which enters dn's and n's terms at most four times: 16 U of the terms' sizes, and
    of their absolute sums in the weights' gradients."""
    g = torch.Generator(device="cuda").manual_seed(C)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, res, gate, dout, dh = (r(9, C) for _ in range(5))
    pre, sc, pw = (1 + 0.3 * r(C) for _ in range(3))
    f = 2.0 ** k

    def run(f):
        # with a norm after the block its output does not scale, alpha does
        kw = dict(gate=gate, scale=sc, post_weight=pw if post else None, eps=0.0,
                  residual_scale=f if post else 1.0)
        xs = x if post else x * f
        out, h = binding.block_norm_fwd(xs, res * f, pre, **kw)
        b = binding.block_norm_bwd(xs, res * f, pre, dout, dh / f, **kw)
        b["out"], b["residual"], b["h"] = out, b["residual"] * f, h / f
        if not post:
            b["x"] = b["x"] * f
        return b

    one, other = run(1.0), run(f)
    torch.cuda.synchronize()
    d = lambda t: t.double()  # noqa: E731
    h = d(one["h"])
    r2 = (h * h).mean(1, keepdim=True).rsqrt()
    n, dn = (h * r2).abs(), (d(dout) * d(pre)).abs()
    size = r2 * (dn + n * (dn * n).mean(1, keepdim=True)) + d(dh).abs()
    act = torch.sigmoid(d(gate))
    m = d(x) * (d(x) * d(x)).mean(1, keepdim=True).rsqrt() if post else d(x)
    p = (m * d(pw) if post else m).abs()
    dp = size * d(sc).abs() * act
    dm = (dp * d(pw).abs()) if post else dp
    r1 = (d(x) * d(x)).mean(1, keepdim=True).rsqrt() if post else 1.0
    sizes = {"out": d(one["out"]).abs(), "h": h.abs(), "residual": size,
             "gate": size * d(sc).abs() * p * act * (1 - act),
             "x": r1 * (dm + m.abs() * (dm * m.abs()).mean(1, keepdim=True)) if post else dp,
             "pre_weight": (d(dout).abs() * n).sum(0), "scale": (size * p * act).sum(0)}
    if post:
        sizes["post_weight"] = (dp * m.abs()).sum(0)
    for name, s in sizes.items():
        err = (d(one[name]) - d(other[name])).abs()
        assert bool((err <= 16 * U * s).all()), (name, float((err / s).max()))


def test_block_norm_no_rows():
    x = torch.empty((0, 512), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, device="cuda")
    out, h = binding.block_norm_fwd(x, x, w)
    g = binding.block_norm_bwd(x, x, w, x, post_weight=w, scale=w)
    torch.cuda.synchronize()
    assert out.shape == h.shape == (0, 512)
    for k in ("pre_weight", "post_weight", "scale"):
        assert not g[k].any()


def test_block_norm_argument_checks():
    d, kw, dtype, rdt = draw("sigmoid")
    e = device(d)
    for bad in (dict(residual=e["residual"].half()), dict(residual=e["residual"][:5]),
                dict(pre_weight=e["pre"].bfloat16()), dict(gate=e["gate"].float()),
                dict(x=e["x"].t()), dict(scale=e["pre"][:5]), dict(gate_activation="tanh"),
                dict(out=e["x"].float()), dict(post_weight=e["pre"].cpu())):
        with pytest.raises(ValueError):
            binding.block_norm_fwd(**{**dict(x=e["x"], residual=e["residual"], pre_weight=e["pre"]), **bad})
    for kw in (dict(eps=-1.0), dict(residual_scale=float("nan"))):
        with pytest.raises(binding.SsdError) as err:
            binding.block_norm_fwd(e["x"], e["residual"], e["pre"], **kw)
        assert err.value.code == binding.SSD_ERR_INVALID_ARG
