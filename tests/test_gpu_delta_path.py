"""A gated-delta layer's operators run together, as a program uses them (GPU): short
convolution, norm of queries and keys, gated delta rule, gated norm; a prompt, then one token
at a time; packed prompts; forward, then backward; on graphs.

The projections are plain matrix products in fp32 outside the library.
"""
import numpy as np
import pytest
import torch

from oracle import delta, layer
from oracle.gated_norm import gated_rmsnorm_bwd, gated_rmsnorm_fwd
from state_space_model_ssd_amd import binding
from tests.helpers import f64, rel_l2

pytestmark = pytest.mark.gpu

H, P, N, G, K = 4, 32, 64, 2, 4
DI, GN, DM = H * P, G * N, 48
C = DI + 2 * GN
ROW = DI + C + 2 * H                              # z | v | k | q | g | beta
SCALE = N ** -0.5
# relative L2 in fp32: the layer's four operators are held to 1e-5 each, in the backward to 1e-4
# (the delta rule) and some 1e-6, twice that for its gradients through the norm
TOL, TOL_BWD = 4e-5, 2e-4


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(win=r(DM, ROW) / DM ** 0.5, wout=r(DI, DM) / DI ** 0.5, cw=r(C, K) * 0.5, cb=r(C) * 0.1,
                gnw=1 + 0.1 * r(DI), qw=1 + 0.1 * r(N), kw=1 + 0.1 * r(N), A=-torch.exp(0.3 * r(H)))


def gates(ga, be, A):
    soft = torch.nn.functional.softplus(ga)
    return (A * soft).contiguous(), torch.sigmoid(be).contiguous()


def front(x, w):
    return (x @ w["win"]).split((DI, C, H, H), -1)


def prompt(x, w, cu=None, conv0=None, S0=None):
    b, T, _ = x.shape
    z, vkq, ga, be = front(x, w)
    v, k, q, conv = binding.conv_fwd(vkq, w["cw"], w["cb"], splits=(DI, GN, GN), initial_states=conv0, cu_seqlens=cu)
    qn, kn = binding.qk_norm_fwd(q.view(b, T, G, N), k.view(b, T, G, N), norm="l2")
    g, beta = gates(ga, be, w["A"])
    y, S, _ = binding.delta_fwd(qn, kn, v.view(b, T, H, P), g, beta, initial_states=S0, cu_seqlens=cu)
    o = binding.gated_norm_fwd(y.view(b, T, DI), z.contiguous(), w["gnw"], DI)
    return o @ w["wout"], conv, S


def token(x, w, conv, S, slots=None):
    b = x.shape[0]
    z, vkq, ga, be = front(x, w)
    v, k, q = binding.conv_step(vkq, conv, w["cw"], w["cb"], splits=(DI, GN, GN), slots=slots)
    qn, kn = binding.qk_norm_fwd(q.view(b, G, N), k.view(b, G, N), norm="l2")
    y = binding.delta_step(qn, kn, v.view(b, H, P), *gates(ga, be, w["A"]), S, slots=slots)
    return binding.gated_norm_fwd(y.view(b, DI), z.contiguous(), w["gnw"], DI) @ w["wout"]


def cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def oracle_prompt(x, w):
    f = {k: f64(v) for k, v in w.items()}
    b, T, _ = x.shape
    zx = f64(x) @ f["win"]
    z, vkq, ga, be = np.split(zx, np.cumsum((DI, C, H)), -1)
    o, conv, _ = layer.conv_fwd(vkq, w["cw"], w["cb"])
    v, k, q = o[..., :DI], o[..., DI:DI + GN], o[..., DI + GN:]
    qn, kn = (delta.head_norm_fwd(t.reshape(b, T, G, N), norm="l2") for t in (q, k))
    g, beta = f["A"] * np.logaddexp(0, ga), 1 / (1 + np.exp(-be))
    y, S, _, _ = delta.delta_fwd(qn, kn, v.reshape(b, T, H, P), g, beta, SCALE)
    on, _ = gated_rmsnorm_fwd(y.reshape(b * T, DI), z.reshape(b * T, DI), f["gnw"], 1e-5, DI)
    return on.reshape(b, T, DI) @ f["wout"], conv, S


def draw(b, T, seed=1):
    return torch.randn((b, T, DM), generator=torch.Generator().manual_seed(seed))


def test_prompt_then_tokens_against_the_oracle():
    w, x = weights(), draw(3, 100)
    ref, conv_ref, S_ref = oracle_prompt(x, w)
    wd, xd = cuda(w), x.cuda()
    out, conv, S = prompt(xd[:, :70].contiguous(), wd)
    outs = [token(xd[:, t].contiguous(), wd, conv, S) for t in range(70, 100)]
    got = torch.cat((out, torch.stack(outs, 1)), 1)
    assert rel_l2(got, ref) <= TOL and rel_l2(conv, conv_ref) <= TOL and rel_l2(S, S_ref) <= TOL


def test_a_prompt_in_two_parts():
    w, x = weights(), draw(2, 150)
    wd, xd = cuda(w), x.cuda()
    whole, conv, S = prompt(xd, wd)
    a, c1, s1 = prompt(xd[:, :77].contiguous(), wd)
    b, c2, s2 = prompt(xd[:, 77:].contiguous(), wd, conv0=c1, S0=s1)
    assert rel_l2(torch.cat((a, b), 1), whole) <= 2 * TOL and rel_l2(s2, S) <= 2 * TOL and rel_l2(c2, conv) <= 2 * TOL


def test_packed_prompts_then_tokens_by_slot():
    """Prompts of several lengths packed, their states into a cache of more slots, then tokens
    of some of them in another order, with padding."""
    w, lens = weights(), [1, 70, 0, 129]
    wd = cuda(w)
    xs = [draw(1, n + 5, seed=10 + i) for i, n in enumerate(lens)]
    refs = [oracle_prompt(x, w) for x in xs]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    pack = torch.cat([x[:, :n] for x, n in zip(xs, lens)], 1).cuda()
    out, conv, S = prompt(pack, wd, cu=cu.cuda())
    for i, n in enumerate(lens):
        if n:
            assert rel_l2(out[0, cu[i]:cu[i + 1]], refs[i][0][0, :n]) <= TOL
    where = [5, 0, 3, 2]
    cc = torch.randn((6,) + conv.shape[1:]).cuda()
    cs = torch.randn((6,) + S.shape[1:]).cuda()
    cc[where], cs[where] = conv, S
    slots = torch.tensor([3, -1, 5, 2, 0], dtype=torch.int32).cuda()
    order = [2, None, 0, 3, 1]
    for t in range(5):
        x = torch.stack([draw(1, 1, 77)[0, 0] if i is None else xs[i][0, lens[i] + t] for i in order]).cuda()
        got = token(x, wd, cc, cs, slots)
        for row, i in enumerate(order):
            if i is not None:
                assert rel_l2(got[row], refs[i][0][0, lens[i] + t]) <= 2 * TOL, (t, i)
    for i in range(4):
        assert rel_l2(cs[where[i]], refs[i][2][0]) <= TOL


def test_backward_against_the_oracle():
    """The gradient of the projection's output, made by each operator's backward in turn, the
    columns of q, k and v in one row of it."""
    w, x = weights(), draw(2, 90)
    wd, xd = cuda(w), x.cuda()
    b, T = 2, 90
    dout = torch.randn((b, T, DI), generator=torch.Generator().manual_seed(3))
    z, vkq, ga, be = front(xd, wd)
    zc = z.contiguous()
    v, k, q, _ = binding.conv_fwd(vkq, wd["cw"], wd["cb"], splits=(DI, GN, GN))
    q4, k4, v4 = q.view(b, T, G, N), k.view(b, T, G, N), v.view(b, T, H, P)
    norm = dict(q_weight=wd["qw"], k_weight=wd["kw"], norm="l2")
    qn, kn = binding.qk_norm_fwd(q4, k4, **norm)
    g, beta = gates(ga, be, wd["A"])
    y, _, _ = binding.delta_fwd(qn, kn, v4, g, beta)
    dy, dz, dgnw = binding.gated_norm_bwd(y.view(b, T, DI), zc, wd["gnw"], dout.cuda(), DI)[:3]
    d = binding.delta_bwd(qn, kn, v4, g, beta, dy.view(b, T, H, P))
    n = binding.qk_norm_bwd(q4, k4, d["q"], d["k"], **norm)
    c = binding.conv_bwd(vkq, wd["cw"], (d["v"].view(b, T, DI), n["k"].view(b, T, GN), n["q"].view(b, T, GN)),
                         wd["cb"], splits=(DI, GN, GN))

    f = {m: f64(t) for m, t in w.items()}
    oz, ovkq, oga, obe = np.split(f64(x) @ f["win"], np.cumsum((DI, C, H)), -1)
    o = layer.conv_fwd(ovkq, w["cw"], w["cb"])[0]
    ov, ok, oq = o[..., :DI], o[..., DI:DI + GN], o[..., DI + GN:]
    oq, ok = oq.reshape(b, T, G, N), ok.reshape(b, T, G, N)
    oqn, okn = delta.head_norm_fwd(oq, w["qw"], "l2"), delta.head_norm_fwd(ok, w["kw"], "l2")
    og, ob = f["A"] * np.logaddexp(0, oga), 1 / (1 + np.exp(-obe))
    oy = delta.delta_fwd(oqn, okn, ov.reshape(b, T, H, P), og, ob, SCALE)[0]
    res = gated_rmsnorm_bwd(oy.reshape(b * T, DI), oz.reshape(b * T, DI), f["gnw"], 1e-5, DI, f64(dout).reshape(b * T, DI))
    r = delta.delta_bwd(oqn, okn, ov.reshape(b, T, H, P), og, ob, res[0].reshape(b, T, H, P), SCALE)
    rq, rqw = delta.head_norm_bwd(oq, r["q"], w["qw"], "l2")
    rk, rkw = delta.head_norm_bwd(ok, r["k"], w["kw"], "l2")
    rc = layer.conv_bwd(ovkq, w["cw"], np.concatenate((r["v"].reshape(b, T, DI), rk.reshape(b, T, GN), rq.reshape(b, T, GN)), -1),
                        w["cb"])
    for what, got, ref in (("g", d["g"], r["g"]), ("beta", d["beta"], r["beta"]), ("q_weight", n["q_weight"], rqw),
                           ("k_weight", n["k_weight"], rkw), ("x", c["x"], rc["x"]), ("weight", c["weight"], rc["weight"]),
                           ("z", dz, res[1])):
        assert rel_l2(got, np.asarray(ref).reshape(got.shape)) <= TOL_BWD, what


def test_tokens_in_a_graph():
    w, x = weights(), draw(3, 60)
    wd, xd = cuda(w), x.cuda()
    _, conv, S = prompt(xd[:, :50].contiguous(), wd)
    gc, gs, buf = conv.clone(), S.clone(), xd[:, 50].contiguous()
    token(buf, wd, conv.clone(), S.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(buf, wd, gc, gs)
    gc.copy_(conv)
    gs.copy_(S)
    for t in range(50, 60):
        buf.copy_(xd[:, t])
        graph.replay()
        torch.cuda.synchronize()
        want = token(xd[:, t].contiguous(), wd, conv, S)
        assert rel_l2(out, want) <= 1e-6 and torch.equal(gc, conv) and rel_l2(gs, S) <= 1e-6, t
