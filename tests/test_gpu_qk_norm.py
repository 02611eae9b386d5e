"""The norm of queries and keys with the rotation on the GPU, against the 64-bit formula.

Bounds, with U = 2^-24: the sum of squares (at most 8 in a lane and 6 exchanges) and the root
24 U, as in the norms around a block.  An angle is rounded to fp32 as a part of a half turn
(pi 2^-25 < 2 U) and to fp64 before (2^-51 of it), its sine and cosine within 4 U: ECS.  The
backward adds 40 U for each dot product, and for a weight's gradient one U for every addition
on the way of a term: 32 tiles of tokens in one register, the registers of a workgroup, and
the partial rows."""
import numpy as np
import pytest
import torch

from oracle import delta
from state_space_model_ssd_amd import binding
from tests.delta_cases import DT
from tests.helpers import f64
from tests.layer_bounds import RND, TINY, U, check

pytestmark = pytest.mark.gpu

E = 24 * U


def inputs(lead=(9,), Hq=4, Hk=2, D=64, R=None, dtype="bf16", weights=True, seed=0, far=False):
    r = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    R = D // 2 if R is None else R
    x = dict(q=2 * rn(*lead, Hq, D), k=0.5 * rn(*lead, Hk, D), dq=rn(*lead, Hq, D), dk=rn(*lead, Hk, D))
    x = {n: v.to(DT[dtype]) for n, v in x.items()}
    x["wq"], x["wk"] = (1 + 0.3 * rn(D), 1 + 0.3 * rn(D)) if weights else (None, None)
    x["pos"] = x["freq"] = None
    if R:
        hi = 2 ** 31 - 1 if far else 4096
        x["pos"] = torch.randint(-hi if far else 0, hi, lead, generator=r).to(torch.int32)
        x["freq"] = 10000.0 ** (-torch.arange(R) / R)
    return x


def on(d):
    return {n: (None if v is None else v.cuda()) for n, v in d.items()}


def pairs(R, interleaved):
    return (np.s_[..., 0:2 * R:2], np.s_[..., 1:2 * R:2]) if interleaved else (np.s_[..., :R], np.s_[..., R:2 * R])


def turned(x, ex, pos, freq, interleaved, back=False):
    """A bound for the turned values, of values x with errors ex."""
    if pos is None:
        return ex
    cos, sin = delta.turns(pos, freq)
    ecs = 6 * U + 2.0 ** -51 * np.abs(f64(pos)[..., None, None] * f64(freq))
    x, e = np.abs(x), ex.copy()
    a, b = pairs(freq.numel(), interleaved)
    c, s = np.abs(cos), np.abs(sin)
    e[a] = ex[a] * c + ex[b] * s + (x[a] + x[b]) * ecs + 3 * U * (x[a] * c + x[b] * s)
    e[b] = ex[b] * c + ex[a] * s + (x[a] + x[b]) * ecs + 3 * U * (x[b] * c + x[a] * s)
    return e


def check_fwd(got, x, norm="rms", eps=1e-6, interleaved=False):
    for name, w, out in (("q", "wq", got[0]), ("k", "wk", got[1])):
        ref = delta.head_norm_fwd(x[name], x[w], norm, eps, x["pos"], x["freq"], interleaved)
        n = delta.head_norm_fwd(x[name], x[w], norm, eps)
        tol = turned(n, (E + 2 * U) * np.abs(n), x["pos"], x["freq"], interleaved)
        dt = "bf16" if x["q"].dtype == torch.bfloat16 else "f32"
        assert out.is_contiguous() and out.dtype == x["q"].dtype
        check(out, ref, tol + RND[dt] * np.abs(ref) + TINY, name)


def check_bwd(got, x, norm="rms", eps=1e-6, interleaved=False):
    dt = "bf16" if x["q"].dtype == torch.bfloat16 else "f32"
    for name, w in (("q", "wq"), ("k", "wk")):
        do = f64(x["d" + name])
        ref, rw = delta.head_norm_bwd(x[name], x["d" + name], x[w], norm, eps, x["pos"], x["freq"], interleaved)
        xs = f64(x[name])
        r = delta._scale_of(xs, norm, eps)
        n = np.abs(xs * r)
        d, ed = do, np.zeros_like(do)
        if x["pos"] is not None:
            cos, sin = delta.turns(x["pos"], x["freq"])
            d = delta.rotate(do, cos, -sin, interleaved)
            ed = turned(do, ed, x["pos"], x["freq"], interleaved)
        d = np.abs(d)
        wt = np.abs(f64(x[w])) if x[w] is not None else np.ones(xs.shape[-1])
        dn, edn = d * wt, ed * wt + U * d * wt
        mean = (lambda v: v.mean(-1, keepdims=True)) if norm == "rms" else (lambda v: v.sum(-1, keepdims=True))
        dot = mean(dn * n)
        tol = r * (edn + n * mean(edn * n + (E + 40 * U) * dn * n) + 2 * E * n * dot + (E + 4 * U) * (dn + n * dot))
        check(got[name], ref, tol + RND[dt] * np.abs(ref) + TINY, "d" + name)
        dw = got[name + "_weight"]
        if x[w] is None:
            assert dw is None
            continue
        rows = int(np.prod(xs.shape[:-1]))
        heads = x["q"].shape[-2] + x["k"].shape[-2]
        adds = min(rows, 32 * 4 * heads) + rows // (32 * heads) // 32 + 256 + 32
        ax = tuple(range(xs.ndim - 1))
        check(dw, rw, (ed * n + E * d * n).sum(ax) + adds * U * (d * n).sum(ax) + U * np.abs(rw) + TINY, "dw" + name)


def run(x, **kw):
    d = on(x)
    a = dict(q_weight=d["wq"], k_weight=d["wk"], positions=d["pos"], inv_freq=d["freq"], **kw)
    return binding.qk_norm_fwd(d["q"], d["k"], **a), binding.qk_norm_bwd(d["q"], d["k"], d["dq"], d["dk"], **a)


SHAPES = [  # lead, Hq, Hk, D, R
    ((1,), 1, 1, 1, 0), ((5,), 2, 1, 2, 1), ((2, 3), 3, 2, 7, 2), ((9,), 4, 2, 64, 32), ((3, 5), 16, 16, 128, 64),
    ((7,), 8, 1, 256, 128), ((33,), 5, 3, 80, 20), ((2, 17), 12, 4, 100, 50), ((40,), 1, 2, 33, 16), ((6,), 3, 3, 9, 4),
    ((1100,), 2, 1, 64, 32), ((4500,), 3, 1, 16, 3), ((0,), 2, 2, 32, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[0] + s[1:])))
def test_norm(shape, dtype):
    lead, Hq, Hk, D, R = shape
    for i, (norm, inter, w) in enumerate((("rms", False, True), ("l2", True, False), ("l2", False, True), ("rms", True, True))):
        x = inputs(lead, Hq, Hk, D, R, dtype, weights=w, seed=i)
        fwd, bwd = run(x, norm=norm, interleaved=inter)
        check_fwd(fwd, x, norm, interleaved=inter)
        check_bwd(bwd, x, norm, interleaved=inter)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_rotation_and_with_one_weight(norm, dtype):
    x = inputs(R=0, dtype=dtype)
    x["wk"] = None
    fwd, bwd = run(x, norm=norm, eps=1e-2)
    check_fwd(fwd, x, norm, 1e-2)
    check_bwd(bwd, x, norm, 1e-2)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    x = inputs((50,), far=True, dtype="f32")
    x["pos"][:3] = torch.tensor([0, 2 ** 31 - 1, -2 ** 31])
    fwd, bwd = run(x, interleaved=interleaved)
    check_fwd(fwd, x, interleaved=interleaved)
    check_bwd(bwd, x, interleaved=interleaved)


def test_more_tokens_than_a_row_of_the_grid():
    """2^20 tokens, four a workgroup: the same as their parts."""
    n, cut = 2 ** 20 + 5, 2 ** 20 - 3
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn((n, 64, 8), device="cuda", generator=g).bfloat16()
    k = torch.randn((n, 1, 8), device="cuda", generator=g).bfloat16()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freq = torch.tensor([1.0, 0.1], device="cuda")
    whole = binding.qk_norm_fwd(q, k, positions=pos, inv_freq=freq)
    for at in (slice(cut, n), slice(0, 2000)):
        part = binding.qk_norm_fwd(q[at], k[at], positions=pos[at], inv_freq=freq)
        assert torch.equal(whole[0][at], part[0]) and torch.equal(whole[1][at], part[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_and_tiny_rows(dtype):
    x = inputs(dtype=dtype)
    x["q"][0], x["k"][1], x["q"][2] = 0, 0, x["q"][2] * 2.0 ** -40
    for norm in ("rms", "l2"):
        fwd, bwd = run(x, norm=norm)
        check_fwd(fwd, x, norm)
        check_bwd(bwd, x, norm)
        assert not fwd[0][0].any() and not fwd[1][1].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 33])
def test_columns_of_one_row(D, dtype):
    """q and k as columns of the projection's rows, their gradients as columns of its gradient;
    the columns between stay."""
    x = inputs((2, 11), 4, 2, D, D // 2, dtype)
    wide = torch.full((2, 11, 6 * D + 5), 3.0, dtype=DT[dtype], device="cuda")
    dwide = torch.full_like(wide, 3.0)
    cut = lambda t: (t[..., 2:2 + 4 * D].unflatten(-1, (4, D)), t[..., 3 + 4 * D:3 + 6 * D].unflatten(-1, (2, D)))  # noqa: E731
    d = on(x)
    q, k = cut(wide)
    q.copy_(d["q"])
    k.copy_(d["k"])
    kept = wide.clone()
    a = dict(q_weight=d["wq"], k_weight=d["wk"], positions=d["pos"], inv_freq=d["freq"])
    check_fwd(binding.qk_norm_fwd(q, k, **a), x)
    dq, dk = cut(dwide)
    got = binding.qk_norm_bwd(q, k, d["dq"], d["dk"], **a, dq=dq, dk=dk)
    assert got["q"] is dq and got["k"] is dk
    check_bwd(got, x)
    assert torch.equal(wide, kept)
    for c in (0, 1, 2 + 4 * D, 3 + 6 * D, 4 + 6 * D):
        assert bool((dwide[..., c] == 3).all())


def test_backward_against_differences():
    x = inputs((3,), 2, 1, 10, 4, "f32")
    _, got = run(x, norm="l2", interleaved=True)
    r = np.random.default_rng(0)

    def value(y):
        tot = 0.0
        for n, w in (("q", "wq"), ("k", "wk")):
            o = delta.head_norm_fwd(y[n], y[w], "l2", 1e-6, x["pos"], x["freq"], True)
            tot += float(np.sum(o * f64(x["d" + n])))
        return tot
    base = {n: f64(x[n]) for n in ("q", "k", "wq", "wk")}
    for n, name in (("q", "q"), ("k", "k"), ("wq", "q_weight"), ("wk", "k_weight")):
        u, h = r.standard_normal(base[n].shape), 1e-6
        num = (value(dict(base, **{n: base[n] + h * u})) - value(dict(base, **{n: base[n] - h * u}))) / (2 * h)
        g = f64(got[name])
        assert abs(num - np.sum(g * u)) <= 1e-5 * (1 + np.sum(np.abs(g * u))), n


@pytest.mark.parametrize("D,Hq", [(128, 4), (16, 1)])
def test_weights_over_many_tokens(D, Hq):
    """Sums over 200000 tokens of equal sign lose no more than short ones."""
    T = 200000
    q = torch.ones((T, Hq, D), device="cuda")
    k = torch.ones((T, 1, D), device="cuda")
    w = torch.ones(D, device="cuda")
    got = binding.qk_norm_bwd(q, k, q, k, w, w, eps=0.0)
    for n, m in (("q_weight", T * Hq), ("k_weight", T)):
        assert float((got[n] / m - 1).abs().max()) <= 2.0 ** -16, n


def test_same_bits_twice_and_workspace_as_found():
    x = on(inputs((3000,), 8, 2, 64, 32))
    a = dict(q_weight=x["wq"], k_weight=x["wk"], positions=x["pos"], inv_freq=x["freq"])
    one = binding.qk_norm_bwd(x["q"], x["k"], x["dq"], x["dk"], **a)
    two = binding.qk_norm_bwd(x["q"], x["k"], x["dq"], x["dk"], **a, workspace=torch.full_like(one["workspace"], 255))
    for n in ("q", "k", "q_weight", "k_weight"):
        assert torch.equal(one[n], two[n]), n


def test_infinities_and_nan_stay_in_their_rows():
    x = on(inputs((20,), 4, 2, 64, 32))
    a = dict(q_weight=x["wq"], k_weight=x["wk"], positions=x["pos"], inv_freq=x["freq"])
    want = binding.qk_norm_fwd(x["q"], x["k"], **a)
    x["q"][3, 1, 7], x["k"][5, 0, 0] = float("inf"), float("nan")
    got = binding.qk_norm_fwd(x["q"], x["k"], **a)
    assert got[0][3, 1].isnan().any() and got[1][5, 0].isnan().all()
    for g, w, at in ((got[0], want[0], (3, 1)), (got[1], want[1], (5, 0))):
        keep = torch.ones_like(g, dtype=torch.bool)
        keep[at] = False
        assert torch.equal(g[keep], w[keep])


def test_in_a_graph_on_a_stream_of_its_own():
    x = on(inputs((300,), 4, 2, 64, 32))
    a = dict(q_weight=x["wq"], k_weight=x["wk"], positions=x["pos"], inv_freq=x["freq"])

    def both():
        return binding.qk_norm_fwd(x["q"], x["k"], **a), binding.qk_norm_bwd(x["q"], x["k"], x["dq"], x["dk"], **a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd, bwd = both()
    for i in range(3):
        y = on(inputs((300,), 4, 2, 64, 32, seed=5 + i))
        for n, v in y.items():
            x[n].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        f, b = both()
        assert torch.equal(fwd[0], f[0]) and torch.equal(fwd[1], f[1])
        for n in ("q", "k", "q_weight", "k_weight"):
            assert torch.equal(bwd[n], b[n]), (i, n)


def test_refusals():
    x = on(inputs())
    bad = [dict(k=x["k"].float()), dict(k=x["k"][:5]), dict(k=x["k"][..., :32]), dict(q=x["q"].cpu()),
           dict(q=x["q"].transpose(0, 1)), dict(q_weight=x["wq"].bfloat16()), dict(q_weight=x["wq"][:32]),
           dict(positions=x["pos"]), dict(inv_freq=x["freq"]), dict(positions=x["pos"].long(), inv_freq=x["freq"]),
           dict(positions=x["pos"][:4], inv_freq=x["freq"]),
           dict(positions=x["pos"], inv_freq=torch.ones(33, device="cuda")), dict(norm="max"), dict(eps=-1.0),
           dict(outs=(x["q"], x["k"])), dict(outs=(x["dq"].float(), x["dk"]))]
    for kw in bad:
        a = dict(dict(q=x["q"], k=x["k"]), **kw)
        with pytest.raises((ValueError, binding.SsdError)):
            binding.qk_norm_fwd(a.pop("q"), a.pop("k"), **a)
    for kw in (dict(dq_out=x["dq"].float()), dict(dk_out=x["dk"][:4]), dict(dq=x["q"]), dict(dk=x["dk"])):
        a = dict(dict(dq_out=x["dq"], dk_out=x["dk"]), **kw)
        with pytest.raises((ValueError, binding.SsdError)):
            binding.qk_norm_bwd(x["q"], x["k"], a.pop("dq_out"), a.pop("dk_out"), **a)
