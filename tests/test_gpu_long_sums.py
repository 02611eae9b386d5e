"""Weight gradients summed over very many tokens (GPU).  A channel's terms are all the
same number, different from channel to channel, so that the roundings of a long chain
of additions all go the same way, and the exact sums are known.

Every addition is off by at most U = 2^-24 of its result, and no partial sum exceeds the
total, so a sum is off by at most U of the total for each addition that a term passes.
"""
import pytest
import torch

from state_space_model_ssd_amd import binding
from tests.layer_bounds import U

pytestmark = pytest.mark.gpu


def constants(C):
    """C numbers of three decimal digits, as fp32 holds them."""
    return torch.tensor([0.1 + 0.013 * (i % 90) for i in range(C)], dtype=torch.float32)


def held(got, want, n, what):
    err = ((got.double().cpu() - want).abs() / want.abs()).max().item()
    print(f"  {what}: {err / U:.1f} U of {n} U", flush=True)
    assert err <= n * U, (what, err / U)


@pytest.mark.parametrize("T,C,K,dtype,nseq,segment,segments", [
    (2 ** 23, 12, 2, "f32", None, 18 * 15, 31),    # short runs of 15 tokens: 547 a wave, 18 a segment
    (2 ** 21, 40, 4, "bf16", None, 5 * 61, 7),     # long runs of 61 tokens: 34 a wave, 5 a segment
    (2 ** 20, 6, 3, "f32", 5000, 19 * 14, 5),      # packed: sequences of 209 and 210 tokens
])
def test_conv_weight_gradients_over_many_tokens(T, C, K, dtype, nseq, segment, segments):
    """Without activation, with x = 1 (and states of 1) every tap's gradient and the bias'
    are the sum of dout: T equal terms, each product with 1 exact.  A term passes one
    addition per token of its segment, one per segment, 4 for the waves, then 8 + 3 + 4
    in the column sums."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    c = constants(C).to(dt)
    x = torch.ones((1, T, C), dtype=dt, device="cuda")
    dout = c.cuda().expand(1, T, C).contiguous()
    w, bias = torch.zeros((C, K), device="cuda"), torch.zeros(C, device="cuda")
    cu = None
    if nseq is not None:
        cu = torch.linspace(0, T, nseq + 1, dtype=torch.float64).round().to(torch.int32).cuda()
    init = torch.ones((nseq or 1, K - 1, C), dtype=dt, device="cuda")
    g = binding.conv_bwd(x, w, [dout, None, None], bias, initial_states=init, cu_seqlens=cu,
                         activation=None)
    torch.cuda.synchronize()
    want, n = c.double() * T, segment + segments + 4 + 15
    held(g["bias"], want, n, "dbias")
    held(g["weight"], want[:, None].expand(C, K), n, "dweight")


@pytest.mark.parametrize("T,C,dtype,residual,segment,segments", [
    (2 ** 23, 4, "f32", "f32", 64, 33),            # one wave a row: 2048 rows and more each
    (2 ** 20 + 3, 260, "bf16", "f32", 64, 9),      # two waves a row, 513 rows each
    (2 ** 20 + 3, 261, "bf16", "bf16", 64, 9),     # the same, rows not whole vectors
    (2 ** 17, 5000, "bf16", "bf16", 64, 9),        # eight waves a row, four vectors a lane
])
def test_block_norm_weight_gradients_over_many_rows(T, C, dtype, residual, segment, segments):
    """x = 1, no residual, weights and scale of 1: both norms' factors are 1 within 4 U (the
    mean's product, half of it through the root, the root's 2), the same in every row.
    dout is c and -c at neighbouring channels, so every sum over a row is 0 exactly: dn =
    dout and dh = dout + dresidual_out = 2 dout.  Then dpre_weight = T dout, dscale = 2 T
    dout and dpost_weight = 2 T dout, every term off by at most 4 + 4 U for the factors and
    8 U for its own operations, the same way in every row.

    A term passes one addition per row of its segment, one per segment, 4 for rows that
    share a workgroup, and 16 + 3 + 16 in the column sums of up to 2048 partial rows.  A
    device with fewer than 256 compute units walks further: twice the segments."""
    dt, rdt = (torch.float32 if d == "f32" else torch.bfloat16 for d in (dtype, residual))
    c = torch.zeros(C)
    c[0::2][:C // 2] = constants(C // 2)
    c[1::2][:C // 2] = -constants(C // 2)
    c = c.to(dt)
    x = torch.ones((T, C), dtype=dt, device="cuda")
    dout = c.cuda().expand(T, C).contiguous()
    w = torch.ones(C, device="cuda")
    dres = dout if rdt == dt else dout.to(rdt)
    g = binding.block_norm_bwd(x, None, w, dout, dres, post_weight=w, scale=w, eps=0.0,
                               residual_dtype=rdt)
    torch.cuda.synchronize()
    keep = c != 0
    n = segment + 2 * segments + 4 + 16 + 3 + 16 + 16
    for k, f in (("pre_weight", 1), ("scale", 2), ("post_weight", 2)):
        held(g[k].cpu()[keep], f * c[keep].double() * T, n, "d" + k)


def close_sums(full, parts, size, n, what):
    """A sum against the fp64 sum of its parts: the same fp32 terms, of absolute sum `size`,
    each through at most n additions on either side."""
    err = (full.double() - sum(p.double() for p in parts)).abs()
    worst = (err / (2 * n * U * size)).max().item()
    print(f"  {what}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1, what


@pytest.mark.parametrize("T,splits,K,dtype,lens,n", [
    (300000, (33, 7, 5), 4, "bf16", (1, 200), 400),          # short runs, vectors that overlap
    (300000, (1, 0, 0), 3, "bf16", (1, 200), 400),           # one channel a thread
    (400000, (65, 3, 0), 2, "f32", (300, 900), 400),
    (500000, (130, 9, 2), 4, "bf16", (1000, 5000), 450),     # long runs
])
def test_conv_backward_of_long_batches_equals_its_parts(T, splits, K, dtype, lens, n):
    """A packed batch of several segments against its sequences in groups that have one:
    the same dx and dinitial_states bit for bit, dweight and dbias as sums."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(T + K)
    cuts = [0]
    while cuts[-1] < T:
        cuts.append(min(T, cuts[-1] + int(torch.randint(*lens, (1,), generator=g))))
    nseq, C = len(cuts) - 1, sum(splits)
    d = torch.Generator(device="cuda").manual_seed(K)
    r = lambda *s: torch.randn(s, generator=d, device="cuda").to(dt)  # noqa: E731
    x, douts = r(1, T, C), [r(1, T, m) for m in splits]
    w, bias = r(C, K).float() * 0.5, r(C).float()
    init, dfin = r(nseq, K - 1, C), r(nseq, K - 1, C)

    def call(a, b):
        cu = torch.tensor([c - cuts[a] for c in cuts[a:b + 1]], dtype=torch.int32, device="cuda")
        s = slice(cuts[a], cuts[b])
        return binding.conv_bwd(x[:, s].contiguous(), w, [o[:, s].contiguous() for o in douts], bias,
                                splits=splits, initial_states=init[a:b].contiguous(),
                                dfinal_states=dfin[a:b].contiguous(), cu_seqlens=cu)

    full = call(0, nseq)
    step = nseq // 25 + 1
    parts = [call(a, min(a + step, nseq)) for a in range(0, nseq, step)]
    again = call(0, nseq)
    torch.cuda.synchronize()
    assert torch.equal(full["x"], torch.cat([p["x"] for p in parts], 1))
    assert torch.equal(full["initial_states"], torch.cat([p["initial_states"] for p in parts]))
    for k in ("x", "weight", "bias", "initial_states"):
        assert torch.equal(full[k], again[k])
    # |dpre| is at most 1.1 |dout|, and a tap's terms are dpre in
    a = torch.cat([o.double().abs() for o in douts], -1)[0] * 1.1
    big = torch.maximum(x.double().abs().amax(1)[0], init.double().abs().amax((0, 1)))
    close_sums(full["bias"], [p["bias"] for p in parts], a.sum(0), n, "dbias")
    close_sums(full["weight"], [p["weight"] for p in parts], (a.sum(0) * big)[:, None], n, "dweight")


@pytest.mark.parametrize("T,C,dtype,residual,gate", [
    (300001, 31, "bf16", "f32", "silu"),           # one wave a row, four rows a workgroup
    (300001, 100, "f32", "f32", None),
    (140001, 300, "bf16", "bf16", "sigmoid"),      # two waves, whole vectors
    (140001, 301, "f32", "f32", "linear"),         # two waves, a tail
    (36001, 2001, "bf16", "f32", "silu"),          # eight waves
    (18001, 4096, "bf16", "bf16", "silu"),         # two vectors a lane
    (18001, 4100, "f32", "f32", None),             # four vectors a lane
])
def test_block_norm_backward_of_many_rows_equals_its_parts(T, C, dtype, residual, gate):
    """Rows of several segments against groups of rows that have one: the same gradients
    per row bit for bit, those of the weights as sums."""
    dt, rdt = (torch.float32 if d == "f32" else torch.bfloat16 for d in (dtype, residual))
    g = torch.Generator(device="cuda").manual_seed(C)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, dout, z = r(T, C).to(dt), r(T, C).to(dt), r(T, C).to(dt) if gate else None
    res, dres = r(T, C).to(rdt), r(T, C).to(rdt)
    pre, post, scale = 1 + 0.3 * r(C), 1 + 0.3 * r(C), 1 + 0.3 * r(C)

    def call(s):
        return binding.block_norm_bwd(x[s], res[s], pre, dout[s], dres[s], gate=z[s] if gate else None,
                                      gate_activation=gate or "linear", post_weight=post, scale=scale,
                                      residual_scale=0.5)

    full, again = call(slice(0, T)), call(slice(0, T))
    step = T // 9 + 1
    parts = [call(slice(a, min(a + step, T))) for a in range(0, T, step)]
    torch.cuda.synchronize()
    for k in ("x", "residual") + (("gate",) if gate else ()):
        assert torch.equal(full[k], torch.cat([p[k] for p in parts])), k
    for k in ("x", "residual", "pre_weight", "post_weight", "scale"):
        assert torch.equal(full[k], again[k]), k
    size = {"pre_weight": 0, "post_weight": 0, "scale": 0}
    for a in range(0, T, step):                    # absolute sums, from the rounded dresidual
        s = slice(a, min(a + step, T))
        xd, dh = x[s].double(), full["residual"][s].double().abs()
        m = xd * (xd * xd).mean(1, keepdim=True).add(1e-5).rsqrt()
        act = torch.ones((), dtype=torch.float64, device="cuda")
        if gate:
            zd = z[s].double()
            act = {"linear": zd, "sigmoid": torch.sigmoid(zd), "silu": zd * torch.sigmoid(zd)}[gate]
        h = res[s].double() + 0.5 * scale.double() * m * post.double() * act
        act = act.abs()
        n = (h * (h * h).mean(1, keepdim=True).add(1e-5).rsqrt()).abs()
        # 1.01: dresidual's and the terms' own roundings
        size["pre_weight"] = size["pre_weight"] + 1.01 * (dout[s].double().abs() * n).sum(0)
        size["scale"] = size["scale"] + 1.01 * (dh * 0.5 * (m * post.double()).abs() * act).sum(0)
        size["post_weight"] = size["post_weight"] + 1.01 * (dh * 0.5 * scale.double().abs() * act * m.abs()).sum(0)
    for k, v in size.items():
        # 64 rows a segment, at most 4 segments, 4 rows, 35 in the column sums
        close_sums(full[k], [p[k] for p in parts], v + 1e-30, 64 + 8 + 4 + 35, "d" + k)


def test_long_sums_in_a_graph():
    """Several segments replayed: the partial rows start anew every time."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    xc, dc, w = r(1, 400000, 6), r(1, 400000, 6), r(6, 4)
    xn, dn, n = r(300000, 40), r(300000, 40), r(40)

    def both():
        a = binding.conv_bwd(xc, w, [dc, None, None], w[:, 0].contiguous())
        b = binding.block_norm_bwd(xn, None, n, dn, post_weight=n, scale=n)
        return [a[k] for k in ("x", "weight", "bias")] + [b[k] for k in ("x", "pre_weight", "post_weight",
                                                                        "scale")]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        both()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            cap = both()
    torch.cuda.synchronize()
    for _ in range(4):
        for t in (xc, dc, xn, dn):
            t.copy_(r(*t.shape))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(cap, both()):
            assert torch.equal(a, b)
