"""The operators of a Mamba-2 layer run together, as a program uses them (GPU):
norm around the block, short convolution, scan, gated norm; a prompt, then one
token at a time; forward, then backward; in HIP graphs and on other streams.

The projections are plain matrix products in fp32 outside the library.
"""
import numpy as np
import pytest
import torch

from oracle import layer
from oracle.backward import ssd_grads
from oracle.gated_norm import gated_rmsnorm_bwd, gated_rmsnorm_fwd
from oracle.recurrence import ssd_recurrence
from state_space_model_ssd_amd import binding
from tests.helpers import rel_l2

pytestmark = pytest.mark.gpu

H, P, N, G, K, L = 4, 32, 16, 2, 4, 64           # fp32 configuration (32, 16, 64)
DI, GN, DM = H * P, G * N, 48
C = DI + 2 * GN
ROW = DI + C + H                                  # z | x | B | C | dt


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(win=r(DM, ROW) / DM ** 0.5, wout=r(DI, DM) / DI ** 0.5, cw=r(C, K) * 0.5, cb=r(C) * 0.1,
                A=-torch.exp(r(H)), D=r(H), dt_bias=r(H) - 2, gnw=1 + 0.1 * r(DI), n1=1 + 0.1 * r(DM),
                n2=1 + 0.1 * r(DM), sc=1 + 0.1 * r(DM))


def prompt(h, x, w, lib=binding):
    """One block over a prompt.  Returns (residual, next input, states)."""
    b, T, _ = x.shape
    hn, res = lib.block_norm_fwd(x, h, w["n1"])
    zx = hn @ w["win"]
    z, xbc, dt = zx.split((DI, C, H), -1)
    xs, B, Cc, conv = lib.conv_fwd(xbc, w["cw"], w["cb"], splits=(DI, GN, GN))
    y, ssm, _ = lib.ssd_fwd(xs.view(b, T, H, P), dt.contiguous(), w["A"], B.view(b, T, G, N),
                            Cc.view(b, T, G, N), L, D=w["D"], dt_bias=w["dt_bias"])
    g = lib.gated_norm_fwd(y.view(b, T, DI), z.contiguous(), w["gnw"], DI)
    out, res2 = lib.block_norm_fwd(g @ w["wout"], res, w["n2"], scale=w["sc"], residual_scale=0.5)
    return res2, out, conv, ssm


def token(h, x, w, conv, ssm, slots=None, lib=binding):
    """The same block for one token per sequence, on its states."""
    b = x.shape[0]
    hn, res = lib.block_norm_fwd(x, h, w["n1"])
    zx = hn @ w["win"]
    z, xbc, dt = zx.split((DI, C, H), -1)
    xs, B, Cc = lib.conv_step(xbc, conv, w["cw"], w["cb"], splits=(DI, GN, GN), slots=slots)
    y = lib.ssd_step(xs.view(b, H, P), dt, w["A"], B.view(b, G, N), Cc.view(b, G, N), ssm, D=w["D"],
                     dt_bias=w["dt_bias"], slots=slots)
    g = lib.gated_norm_fwd(y.view(b, DI), z.contiguous(), w["gnw"], DI)
    out, res2 = lib.block_norm_fwd(g @ w["wout"], res, w["n2"], scale=w["sc"], residual_scale=0.5)
    return res2, out


def cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def draw(b, T, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((b, T, DM), generator=g), torch.randn((b, T, DM), generator=g)


def oracle_prompt(h, x, w):
    f = {k: v.double().numpy() for k, v in w.items()}
    b, T, _ = x.shape
    hn, res = layer.block_norm_fwd(x.reshape(-1, DM), h.reshape(-1, DM), w["n1"])
    zx = hn.reshape(b, T, DM) @ f["win"]
    z, xbc, dt = zx[..., :DI], zx[..., DI:DI + C], zx[..., DI + C:]
    o, conv, _ = layer.conv_fwd(xbc, w["cw"], w["cb"])
    y, ssm = ssd_recurrence(o[..., :DI].reshape(b, T, H, P), dt, f["dt_bias"], f["A"],
                            o[..., DI:DI + GN].reshape(b, T, G, N), o[..., DI + GN:].reshape(b, T, G, N),
                            f["D"])
    g, _ = gated_rmsnorm_fwd(y.reshape(b * T, DI), z.reshape(b * T, DI), f["gnw"], 1e-5, DI)
    out, res2 = layer.block_norm_fwd(g @ f["wout"], res, w["n2"], scale=w["sc"], alpha=0.5)
    return res2.reshape(b, T, DM), out.reshape(b, T, DM), conv, ssm


def test_prompt_then_tokens_against_the_oracle():
    w = weights()
    h, x = draw(3, 90)
    wd, hd, xd = cuda(w), h.cuda(), x.cuda()
    ref = oracle_prompt(h, x, w)
    whole = prompt(hd, xd, wd)
    res, out, conv, ssm = prompt(hd[:, :70].contiguous(), xd[:, :70].contiguous(), wd)
    # the states go to slots of a cache, out of order
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    cc, cs = torch.zeros((6,) + conv.shape[1:], device="cuda"), torch.zeros((6,) + ssm.shape[1:], device="cuda")
    cc[slots.long()], cs[slots.long()] = conv, ssm
    outs = [out] + [token(hd[:, t].contiguous(), xd[:, t].contiguous(), wd, cc, cs, slots)[1][:, None]
                    for t in range(70, 90)]
    torch.cuda.synchronize()
    # fp32 throughout: the projections' sums of 48 and 128 terms and the norms,
    # each some 1e-6 of their size, pass three more operators
    for got, want in zip(whole, ref):
        assert rel_l2(got, want) < 2e-5
    assert rel_l2(torch.cat(outs, 1), ref[1]) < 2e-5
    assert rel_l2(cs[slots.long()], ref[3]) < 2e-5 and rel_l2(cc[slots.long()], ref[2]) < 2e-5
    assert not cs[[1, 3, 5]].any() and not cc[[1, 3, 5]].any()


def test_tokens_in_a_graph_equal_eager_tokens():
    """A decoding step captured once and replayed on changing inputs and slots,
    with eager steps on another cache in between."""
    w = cuda(weights())
    b, steps = 4, 6
    h, x = (v.cuda() for v in draw(b, steps, 3))
    slot_rows = [[0, 1, 2, 3], [3, -1, 5, 0], [1, 1, 4, 2], [-1, -1, -1, -1], [5, 4, 3, 2], [0, 9, 2, 1]]
    g = torch.Generator().manual_seed(9)
    conv = torch.randn((6, K - 1, C), generator=g).cuda()
    ssm = torch.randn((6, H, P, N), generator=g).cuda()
    gc, gs = conv.clone(), ssm.clone()
    hb, xb = h[:, 0].contiguous(), x[:, 0].contiguous()
    slots = torch.full((b,), -1, dtype=torch.int32, device="cuda")   # the warm-up changes no state
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        for _ in range(2):
            token(hb, xb, w, gc, gs, slots)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            gres, gout = token(hb, xb, w, gc, gs, slots)
    torch.cuda.synchronize()
    for t in range(steps):
        hb.copy_(h[:, t])
        xb.copy_(x[:, t])
        slots.copy_(torch.tensor(slot_rows[t], dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        res, out = token(h[:, t].contiguous(), x[:, t].contiguous(), w, conv, ssm, slots)
        torch.cuda.synchronize()
        assert torch.equal(gout, out) and torch.equal(gres, res), t
        assert torch.equal(gc, conv) and torch.equal(gs, ssm), t


def test_backward_of_the_layer_against_the_oracle():
    """conv_bwd behind ssd_bwd behind gated_norm_bwd behind block_norm_bwd."""
    w = weights()
    wd = cuda(w)
    b, T = 2, 70
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    xbc, z, dt, res, do, dh = r(b, T, C), r(b, T, DI), r(b, T, H), r(b, T, DI), r(b, T, DI), r(b, T, DI)
    pre = 1 + 0.1 * r(DI)
    e = {k: v.cuda() for k, v in dict(xbc=xbc, z=z, dt=dt, res=res, do=do, dh=dh, pre=pre).items()}
    xs, B, Cc, _ = binding.conv_fwd(e["xbc"], wd["cw"], wd["cb"], splits=(DI, GN, GN))
    sx, sB, sC = xs.view(b, T, H, P), B.view(b, T, G, N), Cc.view(b, T, G, N)
    y, _, _ = binding.ssd_fwd(sx, e["dt"], wd["A"], sB, sC, L, D=wd["D"], dt_bias=wd["dt_bias"])
    n = binding.gated_norm_fwd(y.view(b, T, DI), e["z"], wd["gnw"], DI)
    gb = binding.block_norm_bwd(n, e["res"], e["pre"], e["do"], e["dh"])
    dy, dz, dgw = binding.gated_norm_bwd(y.view(b, T, DI), e["z"], wd["gnw"], gb["x"], DI)
    gs = binding.ssd_bwd(sx, e["dt"], wd["A"], sB, sC, L, dy.view(b, T, H, P), D=wd["D"],
                         dt_bias=wd["dt_bias"])
    gc = binding.conv_bwd(e["xbc"], wd["cw"], [gs["x"].view(b, T, DI), gs["B"].view(b, T, GN),
                                               gs["C"].view(b, T, GN)], wd["cb"], splits=(DI, GN, GN))
    torch.cuda.synchronize()
    f = {k: v.double().numpy() for k, v in w.items()}
    o, _, _ = layer.conv_fwd(xbc, w["cw"], w["cb"])
    ox, oB, oC = (o[..., :DI].reshape(b, T, H, P), o[..., DI:DI + GN].reshape(b, T, G, N),
                  o[..., DI + GN:].reshape(b, T, G, N))
    ry, _ = ssd_recurrence(ox, dt, f["dt_bias"], f["A"], oB, oC, f["D"])
    flat = lambda v: np.asarray(v, dtype=np.float64).reshape(b * T, -1)  # noqa: E731
    rn, _ = gated_rmsnorm_fwd(flat(ry), flat(z), f["gnw"], 1e-5, DI)
    rb = layer.block_norm_bwd(rn, flat(res), pre, flat(do), flat(dh))
    rdy, rdz, _ = gated_rmsnorm_bwd(flat(ry), flat(z), f["gnw"], 1e-5, DI, rb["x"])
    t64 = lambda v: torch.as_tensor(np.asarray(v, dtype=np.float64))  # noqa: E731
    rs = ssd_grads(t64(ox), dt, w["dt_bias"], w["A"], t64(oB), t64(oC), w["D"],
                   t64(rdy).reshape(b, T, H, P))
    rc = layer.conv_bwd(xbc, w["cw"], np.concatenate([np.asarray(rs[k]).reshape(b, T, -1) for k in ("x", "B", "C")], -1),
                        w["cb"])
    # the scan's gradients are held to 1e-4 in fp32; the others add some 1e-6
    for got, want in ((gb["residual"], rb["residual"].reshape(b, T, DI)), (dz, rdz.reshape(b, T, DI)),
                      (gs["dt"], rs["dt"]), (gc["x"], rc["x"]), (gc["weight"], rc["weight"]),
                      (gc["bias"], rc["bias"])):
        assert rel_l2(got, want) < 2e-4


def test_training_step_in_a_graph():
    """conv and block norm backward captured together, with workspaces made in
    the capture, replayed on changing inputs between eager calls."""
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    w, cw, cb = r(DM), r(C, K), r(C)
    x, xc, res, do = r(130, DM), r(2, 65, C), r(130, DM), r(130, DM)
    dc = [r(2, 65, n) for n in (DI, GN, GN)]

    def both():
        a = binding.conv_bwd(xc, cw, dc, cb, splits=(DI, GN, GN))
        c = binding.block_norm_bwd(x, res, w, do, post_weight=w, scale=w)
        return [a[k] for k in ("x", "weight", "bias")] + [c[k] for k in ("x", "residual", "post_weight",
                                                                         "scale", "pre_weight")]
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        both()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            cap = both()
    torch.cuda.synchronize()
    for rep in range(4):
        for t in (x, xc, res, do, *dc):
            t.copy_(r(*t.shape))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(cap, both()):
            assert torch.equal(a, c), rep


def test_calls_follow_the_current_stream():
    """Two caches stepped on two streams at once equal the same steps in turn."""
    w = cuda(weights())
    h, x = (v.cuda() for v in draw(8, 5, 7))
    g = torch.Generator().manual_seed(2)
    conv = torch.randn((2, 4, K - 1, C), generator=g).cuda()
    ssm = torch.randn((2, 4, H, P, N), generator=g).cuda()
    c1, s1 = conv.clone(), ssm.clone()
    want = [[token(h[4 * i:4 * i + 4, t].contiguous(), x[4 * i:4 * i + 4, t].contiguous(), w, conv[i], ssm[i])
             for t in range(5)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for t in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(token(h[4 * i:4 * i + 4, t].contiguous(), x[4 * i:4 * i + 4, t].contiguous(), w,
                                    c1[i], s1[i]))
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        for (r1, o1), (r2, o2) in zip(a, c):
            assert torch.equal(r1, r2) and torch.equal(o1, o2)
    assert torch.equal(c1, conv) and torch.equal(s1, ssm)
