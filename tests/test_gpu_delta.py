"""The gated delta rule over whole prompts on the GPU, forward and backward, against the
64-bit recurrence one token at a time (and, for the backward, against differences)."""
import numpy as np
import pytest
import torch

from oracle import delta
from state_space_model_ssd_amd import binding
from tests.delta_cases import (check_bwd, check_fwd, dev, draw, draw_grads, inside, unit)
from tests.helpers import f64, rel_l2

pytestmark = pytest.mark.gpu

SHAPES = [  # (b, T, H, G, P, N)
    (1, 1, 4, 2, 16, 32), (2, 2, 2, 1, 64, 128), (1, 63, 3, 3, 48, 64), (1, 64, 4, 1, 32, 128),
    (3, 65, 4, 2, 64, 32), (1, 127, 5, 5, 96, 64), (1, 200, 6, 2, 128, 128), (2, 130, 8, 8, 80, 32),
    (1, 300, 4, 4, 256, 64), (1, 90, 12, 1, 16, 128), (2, 70, 2, 1, 256, 128), (1, 70, 64, 1, 16, 32),
]
IDS = ["x".join(map(str, s)) for s in SHAPES]
TYPES = [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")]


def make(shape, dtype, gate, **kw):
    return draw(*shape, dtype=dtype, gate=gate, **kw)


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape, dtype, gate):
    x = make(shape, dtype, gate)
    check_fwd(binding.delta_fwd(**dev(x)), x, shape[-1] ** -0.5)


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape, dtype, gate):
    x = make(shape, dtype, gate)
    dout, dfin = draw_grads(x)
    got = binding.delta_bwd(**dev(x), dout=dout.cuda(), dfinal_states=dfin.cuda(), scale=0.7)
    check_bwd(got, x, dout, dfin, 0.7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [15, 16, 17, 31, 32, 33])
def test_short_prompts(T, dtype):
    """Around one and two blocks of 16 tokens, rows and packed."""
    x = draw(2, T, 4, 2, 32, 64, dtype)
    check_fwd(binding.delta_fwd(**dev(x)), x, 64 ** -0.5)
    x = draw(1, T, 4, 2, 64, 128, dtype, nseq=3)
    cu = torch.tensor([0, 3, 3, T - 1], dtype=torch.int32)
    check_fwd(binding.delta_fwd(**dev(x), cu_seqlens=cu.cuda()), x, 128 ** -0.5, cu)


# sequences of no, one and many tokens; tokens before the first and behind the last
CUS = [[0, 64, 128], [3, 3, 4, 70, 70, 199], [0, 1, 2, 3, 67, 200], [0, 0, 0], [200, 200], [17, 150],
       [0, 31, 96, 160, 200, 200]]


@pytest.mark.parametrize("dtype,gate,P,N", [("bf16", "f32", 64, 128), ("f32", "f32", 48, 32),
                                            ("bf16", "bf16", 96, 64)])
@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("cu", CUS, ids=lambda c: "-".join(map(str, c)))
def test_packed(cu, init, dtype, gate, P, N):
    x = draw(1, 200, 4, 2, P, N, dtype, gate, nseq=len(cu) - 1, init=init)
    d, c = dev(x), torch.tensor(cu, dtype=torch.int32)
    m = inside(x, c)
    got = binding.delta_fwd(**d, cu_seqlens=c.cuda())
    check_fwd(got, x, N ** -0.5, c)
    assert not f64(got[0].cpu()[~m]).any()                   # zeros in a tensor of the call's own
    kept = torch.full_like(d["v"], 7.0)
    again = binding.delta_fwd(**d, cu_seqlens=c.cuda(), out=kept)
    assert again[0] is kept and bool((kept.cpu()[~m] == 7).all())    # kept in the caller's
    assert torch.equal(kept.cpu()[m], got[0].cpu()[m]) and torch.equal(again[1], got[1])
    dout, dfin = draw_grads(x)
    grads = binding.delta_bwd(**d, cu_seqlens=c.cuda(), dout=dout.cuda(),
                              dfinal_states=None if dfin is None else dfin.cuda())
    check_bwd(grads, x, dout, dfin, N ** -0.5, c)
    # an empty sequence's state passes through, as its gradient does
    for s in range(len(cu) - 1):
        if cu[s] == cu[s + 1]:
            want = d["initial_states"][s] if init else torch.zeros_like(got[1][s])
            assert torch.equal(got[1][s], want)
            if init:
                assert torch.equal(grads["initial_states"][s], dfin[s].cuda())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_is_the_rows(dtype):
    """Equal sequences packed end to end are the rows of a batch, bit for bit."""
    x = draw(3, 128, 4, 2, 64, 64, dtype)
    d = dev(x)
    rows = binding.delta_fwd(**d)
    p = {k: (v if k == "initial_states" else v.reshape(1, 384, *v.shape[2:])) for k, v in d.items()}
    cu = torch.tensor([0, 128, 256, 384], dtype=torch.int32).cuda()
    packed = binding.delta_fwd(**p, cu_seqlens=cu)
    assert torch.equal(rows[0].reshape(-1), packed[0].reshape(-1)) and torch.equal(rows[1], packed[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cut", [1, 63, 64, 65, 150])
def test_states_continue(dtype, cut):
    x = draw(2, 190, 4, 2, 32, 64, dtype)
    a = {k: (v if k == "initial_states" else v[:, :cut].contiguous()) for k, v in x.items()}
    z = {k: (v if k == "initial_states" else v[:, cut:].contiguous()) for k, v in x.items()}
    o1, f1, _ = binding.delta_fwd(**dev(a))
    z = dev(z)
    z["initial_states"] = f1
    o2, f2, _ = binding.delta_fwd(**z)
    check_fwd((torch.cat((o1, o2), 1), f2, None), x, 64 ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["forget", "neg_inf", "keep", "beta0", "beta1", "same_keys", "zero_keys",
                                  "mixed"])
def test_gates_and_keys_at_their_ends(kind, dtype):
    """Decays of nothing and of everything, beta 0 and 1, keys alike or zero."""
    x = draw(1, 150, 4, 2, 32, 64, dtype)
    g, beta, k = x["g"], x["beta"], x["k"]
    if kind == "forget":
        g.fill_(-200.0)
    elif kind == "neg_inf":
        g[:, ::7] = -float("inf")
    elif kind == "keep":
        g.zero_()
    elif kind == "beta0":
        beta.zero_()
    elif kind == "beta1":
        beta.fill_(1.0)
        g.zero_()
    elif kind == "same_keys":
        r = torch.Generator().manual_seed(5)
        k.copy_(unit(k[:, :1].float() + 0.02 * torch.randn(k.shape, generator=r)).to(k.dtype))
        beta.fill_(1.0)
    elif kind == "zero_keys":
        k[:, 20:90] = 0
    else:
        r = torch.Generator().manual_seed(6)
        g.copy_(-torch.exp(3 * torch.randn(g.shape, generator=r)))
        beta.copy_((beta > 0.5).to(beta.dtype))
    check_fwd(binding.delta_fwd(**dev(x)), x, 64 ** -0.5)
    dout, dfin = draw_grads(x)
    got = binding.delta_bwd(**dev(x), dout=dout.cuda(), dfinal_states=dfin.cuda())
    if kind == "neg_inf":                    # the oracle's -inf * 0: its gradient there is 0
        x = dict(x, g=g.clamp_min(-512))
    check_bwd(got, x, dout, dfin, 64 ** -0.5)


@pytest.mark.parametrize("T", [100, 3300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_with_only_one_of_the_states(dtype, T):
    """A gradient of the final states without initial ones, and the other way round."""
    x = draw(1, T, 2, 1, 32, 64, dtype, decay=0.003)
    dout, dfin = draw_grads(x)
    got = binding.delta_bwd(**dev(x), dout=dout.cuda())
    check_bwd(got, x, dout, None, 64 ** -0.5)
    x["initial_states"] = None
    got = binding.delta_bwd(**dev(x), dout=dout.cuda(), dfinal_states=dfin.cuda())
    check_bwd(got, x, dout, dfin, 64 ** -0.5)


def test_no_length_no_sequences():
    for b, T in ((2, 0), (0, 50)):
        x = draw(b, T, 4, 2, 32, 64)
        d = dev(x)
        out, fin, _ = binding.delta_fwd(**d)
        assert out.shape == x["v"].shape and torch.equal(fin, d["initial_states"])
        dfin = torch.randn_like(fin)
        got = binding.delta_bwd(**d, dout=torch.empty_like(out), dfinal_states=dfin)
        assert torch.equal(got["initial_states"], dfin)
        d["initial_states"] = None
        assert not binding.delta_fwd(**d)[1].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_stays_in_its_sequence_and_head(dtype):
    x = draw(1, 200, 4, 4, 32, 64, dtype, nseq=3)
    cu = torch.tensor([0, 70, 140, 200], dtype=torch.int32).cuda()
    d = dev(x)
    clean = binding.delta_fwd(**d, cu_seqlens=cu)
    for name, at in (("v", (0, 100, 1, 3)), ("k", (0, 100, 1, 0)), ("g", (0, 100, 1)), ("beta", (0, 100, 1))):
        bad = {k: v.clone() for k, v in d.items()}
        bad[name][at] = float("nan")
        out, fin, _ = binding.delta_fwd(**bad, cu_seqlens=cu)
        assert out[0, 100:140, 1].isnan().any() and fin[1, 1].isnan().any(), name
        keep = torch.ones_like(out, dtype=torch.bool)
        keep[0, 70:140, 1] = False
        assert torch.equal(out[keep], clean[0][keep]), name
        assert torch.equal(fin[[0, 2]], clean[1][[0, 2]]), name
        assert torch.equal(fin[1, [0, 2, 3]], clean[1][1, [0, 2, 3]]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_twice(dtype):
    x = draw(2, 300, 8, 2, 64, 128, dtype, seed=3)
    d = dev(x)
    dout, dfin = (t.cuda() for t in draw_grads(x))
    a, b = (binding.delta_fwd(**d) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = (binding.delta_bwd(**d, dout=dout, dfinal_states=dfin) for _ in range(2))
    for n in ("q", "k", "v", "g", "beta", "initial_states"):
        assert torch.equal(a[n], b[n]), n


def test_inputs_stay_and_workspace_is_used_as_found():
    x = draw(1, 150, 4, 2, 64, 64)
    d = dev(x)
    before = {k: v.clone() for k, v in d.items()}
    out, fin, ws = binding.delta_fwd(**d)
    dirty = torch.full_like(ws, 255)
    out2, fin2, _ = binding.delta_fwd(**d, workspace=dirty)
    assert torch.equal(out, out2) and torch.equal(fin, fin2)
    dout, dfin = (t.cuda() for t in draw_grads(x))
    got = binding.delta_bwd(**d, dout=dout, dfinal_states=dfin)
    again = binding.delta_bwd(**d, dout=dout, dfinal_states=dfin,
                              workspace=torch.full_like(got["workspace"], 255))
    for n in ("q", "k", "v", "g", "beta", "initial_states"):
        assert torch.equal(got[n], again[n]), n
    for n in before:
        assert torch.equal(before[n], d[n]), n


@pytest.mark.parametrize("dtype,N,P,G", [("f32", 32, 16, 1), ("f32", 128, 48, 2), ("bf16", 64, 32, 2)])
def test_backward_against_differences(dtype, N, P, G):
    """Along random directions, differences of the 64-bit forward: fp32's and pairs' gradients
    to 2^-13 and the rounded ones to the rounding of bf16's operands, of the size that the
    direction's terms have together."""
    x = draw(1, 80, 2, G, P, N, dtype, seed=11)
    dout, dfin = draw_grads(x)
    got = binding.delta_bwd(**dev(x), dout=dout.cuda(), dfinal_states=dfin.cuda(), scale=0.5)
    r = np.random.default_rng(0)
    names = dict(q="q", k="k", v="v", g="g", beta="beta", initial_states="init")
    xd = {n: f64(x[n]) for n in names}
    def value(**ch):
        y = dict(xd, **ch)
        out, fin, _, _ = delta.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], 0.5, y["initial_states"])
        return float(np.sum(out * f64(dout)) + np.sum(fin * f64(dfin)))
    for n in names:
        u, h = r.standard_normal(xd[n].shape), 1e-5
        num = (value(**{n: xd[n] + h * u}) - value(**{n: xd[n] - h * u})) / (2 * h)
        g = f64(got[n])
        exact = dtype == "f32" or n in ("g", "beta", "initial_states")
        tol = (1e-4 if exact else 2e-2) * np.linalg.norm(g) * 4     # a normal direction: within 4 sigma
        assert abs(num - np.sum(g * u)) <= tol, n


def test_gradients_of_the_shared_heads_are_sums():
    """One group of queries and keys for all heads: the sum of what each head gives alone."""
    x = draw(1, 100, 6, 1, 32, 64, "f32")
    dout, dfin = draw_grads(x)
    d, do, df = dev(x), dout.cuda(), dfin.cuda()
    whole = binding.delta_bwd(**d, dout=do, dfinal_states=df)
    parts = {"q": 0, "k": 0}
    for h in range(6):
        one = dict(q=d["q"], k=d["k"], v=d["v"][:, :, h:h + 1].contiguous(),
                   g=d["g"][:, :, h:h + 1].contiguous(), beta=d["beta"][:, :, h:h + 1].contiguous(),
                   initial_states=d["initial_states"][:, h:h + 1].contiguous())
        got = binding.delta_bwd(**one, dout=do[:, :, h:h + 1].contiguous(),
                                dfinal_states=df[:, h:h + 1].contiguous())
        for n in parts:
            parts[n] = parts[n] + got[n].double()
        for n in ("v", "g", "beta"):
            assert rel_l2(whole[n][:, :, h], got[n][:, :, 0]) <= 1e-5
    for n in parts:
        assert rel_l2(whole[n], parts[n]) <= 1e-5, n


def test_a_lone_token_has_no_decay_gradient():
    """Without a state before it, a sequence's first token decays nothing: exactly zero."""
    x = draw(1, 5, 4, 2, 32, 64, init=False, nseq=5)
    cu = torch.arange(6, dtype=torch.int32).cuda()
    got = binding.delta_bwd(**dev(x), dout=torch.randn_like(x["v"]).cuda(), cu_seqlens=cu)
    assert not got["g"].any() and got["beta"].any()


@pytest.mark.parametrize("b,T,H", [(1, 64 * 40, 64), (2, 1500, 48)])
def test_backward_where_the_gates_gradients_are_rounded(b, T, H):
    """bf16 gates over many tokens (more than 65536 tokens times heads) take the variant that
    keeps rounded operands; fp32 gates of the same values the one of pairs."""
    x = draw(b, T, H, H // 16, 32, 32, "bf16", "bf16", seed=4, decay=0.02)
    assert b * T * H > 65536
    dout, dfin = draw_grads(x)
    got = binding.delta_bwd(**dev(x), dout=dout.cuda(), dfinal_states=dfin.cuda())
    check_bwd(got, x, dout, dfin, 32 ** -0.5)
    y = dict(x, g=x["g"].float(), beta=x["beta"].float())
    fine = binding.delta_bwd(**dev(y), dout=dout.cuda(), dfinal_states=dfin.cuda())
    check_bwd(fine, y, dout, dfin, 32 ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_and_heads(dtype):
    """More work than the device has room for at once, in uneven pieces."""
    lens = [(37 * i) % 101 for i in range(40)]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    x = draw(1, int(cu[-1]) + 9, 16, 4, 64, 32, dtype, nseq=40, seed=8)
    check_fwd(binding.delta_fwd(**dev(x), cu_seqlens=cu.cuda()), x, 32 ** -0.5, cu)
    dout, dfin = draw_grads(x)
    got = binding.delta_bwd(**dev(x), cu_seqlens=cu.cuda(), dout=dout.cuda(), dfinal_states=dfin.cuda())
    check_bwd(got, x, dout, dfin, 32 ** -0.5, cu)


@pytest.mark.parametrize("n", [64, 65, 150])
def test_more_sequences_than_a_wave(n):
    """Up to 64 sequences are planned in one launch, more in several; tokens outside cleared."""
    lens = [(11 * i) % 7 + (70 if i == 3 else 0) for i in range(n)]
    cu = torch.tensor(list(np.cumsum([4] + lens)), dtype=torch.int32)
    x = draw(1, int(cu[-1]) + 6, 2, 1, 16, 32, nseq=n, seed=9)
    c = cu.cuda()
    got = binding.delta_fwd(**dev(x), cu_seqlens=c)
    check_fwd(got, x, 32 ** -0.5, cu)
    assert not got[0][:, :4].any() and not got[0][:, -6:].any()
    dout, dfin = draw_grads(x)
    grads = binding.delta_bwd(**dev(x), cu_seqlens=c, dout=dout.cuda(), dfinal_states=dfin.cuda())
    check_bwd(grads, x, dout, dfin, 32 ** -0.5, cu)


def test_long_prompt_of_one_head():
    x = draw(1, 5000, 1, 1, 16, 32, "f32", decay=0.01)
    check_fwd(binding.delta_fwd(**dev(x)), x, 32 ** -0.5)


# few heads and long sequences: cut into segments of 16 chunks or more (at most 64 workgroups of
# 64 values; rows from 32 chunks, packed batches from 64 on)
CUT = [("bf16", 32, 128, None), ("f32", 48, 32, None), ("bf16", 80, 64, [0, 3300, 3300, 3301, 4700]),
       ("f32", 16, 128, [5, 2000, 5900, 6000]), ("bf16", 16, 32, [0, 1024, 5000])]


@pytest.mark.parametrize("dtype,P,N,cu", CUT)
def test_long_sequences_are_cut(dtype, P, N, cu):
    x = draw(1, cu[-1] + 40 if cu else 3300, 2, 1, P, N, dtype, nseq=len(cu) - 1 if cu else None, decay=0.003)
    c = torch.tensor(cu, dtype=torch.int32) if cu else None
    kw = dict(cu_seqlens=c.cuda()) if cu else {}
    check_fwd(binding.delta_fwd(**dev(x), **kw), x, N ** -0.5, c)
    dout, dfin = draw_grads(x)
    got = binding.delta_bwd(**dev(x), **kw, dout=dout.cuda(), dfinal_states=dfin.cuda())
    check_bwd(got, x, dout, dfin, N ** -0.5, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_sequences_that_do_not_decay(dtype):
    """g = 0: what segments hand on is only forgotten where a key comes again."""
    x = draw(1, 12000, 1, 1, 16, 64, dtype)
    x["g"].zero_()
    check_fwd(binding.delta_fwd(**dev(x)), x, 64 ** -0.5)


def test_rows_are_cut_alike():
    """Two rows of equal inputs: cut at the same places, bit for bit, and as a packed pair."""
    x = dev(draw(1, 4224, 2, 1, 32, 64, decay=0.003))
    two = {n: torch.cat((v, v)) for n, v in x.items()}
    out, fin, _ = binding.delta_fwd(**two)
    assert torch.equal(out[0], out[1]) and torch.equal(fin[0], fin[1])
    again = binding.delta_fwd(**two)
    assert torch.equal(again[0], out) and torch.equal(again[1], fin)
    p = {n: (v if n == "initial_states" else v.reshape(1, -1, *v.shape[2:])) for n, v in two.items()}
    packed = binding.delta_fwd(**p, cu_seqlens=torch.tensor([0, 4224, 8448], dtype=torch.int32).cuda())
    assert torch.equal(packed[0].view_as(out), out) and torch.equal(packed[1], fin)


def test_cutting_in_a_graph_follows_the_lengths():
    """Captured where nothing is cut, replayed where the lengths ask for it."""
    d = dev(draw(1, 6400, 2, 1, 32, 64, nseq=4, decay=0.003))
    cu = torch.tensor([0, 1600, 3200, 4800, 6400], dtype=torch.int32).cuda()
    binding.delta_fwd(**d, cu_seqlens=cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, fin, _ = binding.delta_fwd(**d, cu_seqlens=cu)
    for lens in ([0, 1600, 3200, 4800, 6400], [0, 10, 20, 30, 6400], [0, 6400, 6400, 6400, 6400], [7, 3000, 3000, 6000, 6001]):
        cu.copy_(torch.tensor(lens))
        graph.replay()
        torch.cuda.synchronize()
        eager = binding.delta_fwd(**d, cu_seqlens=cu)
        assert torch.equal(out, eager[0]) and torch.equal(fin, eager[1]), lens


@pytest.mark.parametrize("cu", [[0, 6000, 100], [0, -5, 10 ** 9], [4000, 0, 6000], [0, 6000, -1]])
def test_bad_lengths_of_long_batches_stay_in_bounds(cu):
    x = draw(1, 6000, 2, 1, 16, 32, nseq=2)
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    out = torch.full((1, 6128, 2, 16), 5.0, dtype=torch.bfloat16, device="cuda")
    fin = torch.full((4, 2, 16, 32), 5.0, device="cuda")
    binding.delta_fwd(**dev(x), cu_seqlens=c, out=out[:, 64:6064], final_states=fin[1:3])
    torch.cuda.synchronize()
    assert bool((out[:, :64] == 5).all()) and bool((out[:, 6064:] == 5).all())
    assert bool((fin[0] == 5).all()) and bool((fin[3] == 5).all())


@pytest.mark.parametrize("cu", [[0, -5, 64], [0, 100, 50], [0, 50, 10 ** 6], [-3, 20, 64], [2 ** 31 - 1, 0, 1]])
def test_bad_lengths_stay_in_bounds(cu):
    """Lengths that do not rise or pass the tokens are read as far as they make sense: nothing
    outside the arrays is touched, which guard rows around them show."""
    x = draw(1, 64, 4, 2, 32, 64, nseq=2)
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    big = torch.full((1, 192, 4, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, 64:128]
    fin = torch.full((4, 4, 32, 64), 5.0, device="cuda")
    binding.delta_fwd(**dev(x), cu_seqlens=c, out=out, final_states=fin[1:3])
    torch.cuda.synchronize()
    assert bool((big[:, :64] == 5).all()) and bool((big[:, 128:] == 5).all())
    assert bool((fin[0] == 5).all()) and bool((fin[3] == 5).all())


def test_other_stream_and_two_at_once():
    xs = [draw(2, 200, 4, 2, 64, 64, seed=s) for s in (1, 2)]
    ds = [dev(x) for x in xs]
    want = [binding.delta_fwd(**d) for d in ds]
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in ds]
    for d, s in zip(ds, streams):
        with torch.cuda.stream(s):
            got.append(binding.delta_fwd(**d))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("packed", [False, True])
def test_in_a_graph(packed):
    """Forward and backward captured together, replayed on changed inputs and lengths with
    eager calls between."""
    x = draw(1, 200, 4, 2, 64, 64, nseq=3 if packed else None)
    d = dev(x)
    cu = torch.tensor([0, 70, 140, 200], dtype=torch.int32).cuda() if packed else None
    dout, dfin = (t.cuda() for t in draw_grads(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def both():
        out, fin, _ = binding.delta_fwd(**d, cu_seqlens=cu)
        return out, fin, binding.delta_bwd(**d, cu_seqlens=cu, dout=dout, dfinal_states=dfin)
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, fin, grads = both()
    for i in range(4):
        y = dev(draw(1, 200, 4, 2, 64, 64, nseq=3 if packed else None, seed=20 + i))
        for n in y:
            d[n].copy_(y[n])
        if packed:
            cu.copy_(torch.tensor([[0, 70, 140, 200], [5, 5, 6, 150], [0, 64, 64, 100], [0, 1, 2, 3]][i]))
        graph.replay()
        torch.cuda.synchronize()
        eo, ef, eg = both()
        assert torch.equal(out, eo) and torch.equal(fin, ef)
        for n in ("q", "k", "v", "g", "beta", "initial_states"):
            assert torch.equal(grads[n], eg[n]), (i, n)


def test_two_graphs_with_workspaces_of_their_own():
    xs = [draw(1, 150, 4, 2, 32, 64, seed=s) for s in (1, 2)]
    ds, graphs, outs = [dev(x) for x in xs], [], []
    want = [binding.delta_fwd(**d)[:2] for d in ds]
    for d in ds:
        g = torch.cuda.CUDAGraph()
        ws = torch.empty_like(binding.delta_fwd(**d)[2])
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs.append(binding.delta_fwd(**d, workspace=ws))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])


def test_refusals():
    x = dev(draw(1, 64, 4, 2, 32, 64))
    ok = lambda **kw: binding.delta_fwd(**dict(x, **kw))  # noqa: E731
    ok()
    for kw in (dict(k=x["k"][:, :, :, :32]), dict(k=x["k"].float()), dict(v=x["v"][:, :32]),
               dict(v=x["v"].float()), dict(g=x["g"].double()), dict(beta=x["beta"].bfloat16()),
               dict(g=x["g"][:, :32]), dict(initial_states=x["initial_states"].bfloat16()),
               dict(initial_states=x["initial_states"][:, :2]), dict(q=x["q"].cpu()),
               dict(q=x["q"].transpose(1, 2)), dict(v=x["v"].transpose(1, 2)),
               dict(cu_seqlens=torch.tensor([0, 64]).cuda()), dict(scale=float("nan")),
               dict(out=torch.empty_like(x["v"]).float()), dict(out=x["v"]),
               dict(final_states=torch.empty(1, 4, 32, 32, device="cuda")),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, binding.SsdError)):
            ok(**kw)
    with pytest.raises((ValueError, binding.SsdError)):
        binding.delta_bwd(**x, dout=None)
    with pytest.raises((ValueError, binding.SsdError)):
        binding.delta_bwd(**x, dout=torch.empty_like(x["v"]).float())


def test_final_states_may_be_left_out():
    x = dev(draw(1, 100, 4, 2, 32, 64))
    a = binding.delta_fwd(**x)
    b = binding.delta_fwd(**x, return_final_states=False)
    assert b[1] is None and torch.equal(a[0], b[0])
