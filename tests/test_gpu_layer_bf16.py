"""The operators of a Mamba-2 layer run together in bf16 with an fp32 residual stream, as a
layer is trained and served (GPU), for every tap count; tests/test_gpu_layer_path.py does
the same in fp32.

Bound, relative L2 against the fp64 oracle of the whole chain.  A tensor rounded to bf16 is
off by at most 2^-8 of each element.  Between the stream and a result lie the norm's
output, the projection's, the convolution's, the scan's, the gated norm's, the second
projection's and the last norm's: seven roundings, and the scan's own error, 2e-2 by its
tests.  An operator passes an error on by its slope: at most 1.1 for SiLU, about 1 for the
norms and projections, and twice for the gated norm, where y and z both carry it.  So 2 x
(7 x 2^-8 + 2e-2) = 0.095 covers a chain; a wrong row, stride, tap or state is off by 1.
The backward has as many roundings and the same scan bound.
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

TOL = 2 * (7 * 2.0 ** -8 + 2e-2)
H, P, N, G, L = 4, 32, 32, 2, 64                 # bf16 configuration (32, 32, 64)
DI, GN, DM = H * P, G * N, 96
C = DI + 2 * GN
ROW = DI + C + H                                  # z | x | B | C | dt
BF = torch.bfloat16


def weights(K, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(win=(r(DM, ROW) / DM ** 0.5).to(BF), wout=(r(DI, DM) / DI ** 0.5).to(BF),
                cw=r(C, K) * 0.5, cb=r(C) * 0.1, A=-torch.exp(r(H)), D=r(H), dt_bias=r(H) - 2,
                gnw=1 + 0.1 * r(DI), n1=1 + 0.1 * r(DM), n2=1 + 0.1 * r(DM), sc=1 + 0.1 * r(DM))


def rows(x, w):
    """A projection, as a product of two matrices."""
    return (x.reshape(-1, x.shape[-1]) @ w).view(*x.shape[:-1], w.shape[1])


def after(g, res, w):
    """The block's output joins the stream; the next block's input, and the stream."""
    return binding.block_norm_fwd(rows(g, w["wout"]), res, w["n2"], scale=w["sc"], residual_scale=0.5)


def prompt(h, x, w, cu=None):
    b, T, _ = x.shape
    hn, res = binding.block_norm_fwd(x, h, w["n1"])
    z, xbc, dt = rows(hn, w["win"]).split((DI, C, H), -1)
    xs, B, Cc, conv = binding.conv_fwd(xbc, w["cw"], w["cb"], splits=(DI, GN, GN), cu_seqlens=cu)
    y, ssm, _ = binding.ssd_fwd(xs.view(b, T, H, P), dt.float().contiguous(), w["A"],
                                B.view(b, T, G, N), Cc.view(b, T, G, N), L, D=w["D"],
                                dt_bias=w["dt_bias"], cu_seqlens=cu)
    g = binding.gated_norm_fwd(y.view(b, T, DI), z.contiguous(), w["gnw"], DI)
    return after(g, res, w)[0], conv, ssm


def token(h, x, w, conv, ssm, slots):
    b = x.shape[0]
    hn, res = binding.block_norm_fwd(x, h, w["n1"])
    z, xbc, dt = rows(hn, w["win"]).split((DI, C, H), -1)
    xs, B, Cc = binding.conv_step(xbc, conv, w["cw"], w["cb"], splits=(DI, GN, GN), slots=slots)
    y = binding.ssd_step(xs.view(b, H, P), dt, w["A"], B.view(b, G, N), Cc.view(b, G, N), ssm,
                         D=w["D"], dt_bias=w["dt_bias"], slots=slots)
    g = binding.gated_norm_fwd(y.view(b, DI), z.contiguous(), w["gnw"], DI)
    return after(g, res, w)[0]


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
    out, _ = layer.block_norm_fwd(g @ f["wout"], res, w["n2"], scale=w["sc"], alpha=0.5)
    return out.reshape(b, T, DM), conv, ssm


def draw(b, T, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((b, T, DM), generator=g), torch.randn((b, T, DM), generator=g).to(BF)


@pytest.mark.parametrize("K", [2, 3, 4])
def test_prompt_then_tokens(K):
    w = weights(K)
    h, x = draw(3, 90)
    wd, hd, xd = {k: v.cuda() for k, v in w.items()}, h.cuda(), x.cuda()
    ref, rconv, rssm = oracle_prompt(h, x, w)
    whole, wconv, wssm = prompt(hd, xd, wd)
    out, conv, ssm = prompt(hd[:, :70].contiguous(), xd[:, :70].contiguous(), wd)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    cc = torch.zeros((6,) + conv.shape[1:], dtype=BF, device="cuda")
    cs = torch.zeros((6,) + ssm.shape[1:], device="cuda")
    cc[slots.long()], cs[slots.long()] = conv, ssm
    outs = [out] + [token(hd[:, t].contiguous(), xd[:, t].contiguous(), wd, cc, cs, slots)[:, None]
                    for t in range(70, 90)]
    # the same prompts packed into one row
    cu = torch.arange(0, 3 * 90 + 1, 90, dtype=torch.int32, device="cuda")
    packed, pconv, pssm = prompt(hd.view(1, 270, DM), xd.view(1, 270, DM), wd, cu)
    torch.cuda.synchronize()
    for what, got, want in (("prompt", whole, ref), ("tokens", torch.cat(outs, 1), ref),
                            ("packed", packed.view(3, 90, DM), ref), ("conv states", wconv, rconv),
                            ("conv states of the tokens", cc[slots.long()], rconv),
                            ("packed conv states", pconv, rconv), ("scan states", wssm, rssm),
                            ("scan states of the tokens", cs[slots.long()], rssm),
                            ("packed scan states", pssm, rssm)):
        e = rel_l2(got, want)
        print(f"  {what}: {e:.2e} of {TOL:.2e}", flush=True)
        assert e <= TOL, what
    assert not cs[[1, 3, 5]].any() and not cc[[1, 3, 5]].any()


@pytest.mark.parametrize("K", [2, 4])
def test_backward(K):
    w = weights(K)
    wd = {k: v.cuda() for k, v in w.items()}
    b, T = 2, 70
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    xbc, z, do = r(b, T, C).to(BF), r(b, T, DI).to(BF), r(b, T, DI).to(BF)
    dt, res, dh, pre = r(b, T, H), r(b, T, DI), r(b, T, DI), 1 + 0.1 * r(DI)
    e = {k: v.cuda() for k, v in dict(xbc=xbc, z=z, dt=dt, res=res, do=do, dh=dh, pre=pre).items()}
    xs, B, Cc, _ = binding.conv_fwd(e["xbc"], wd["cw"], wd["cb"], splits=(DI, GN, GN))
    sx, sB, sC = xs.view(b, T, H, P), B.view(b, T, G, N), Cc.view(b, T, G, N)
    y, _, _ = binding.ssd_fwd(sx, e["dt"], wd["A"], sB, sC, L, D=wd["D"], dt_bias=wd["dt_bias"])
    n = binding.gated_norm_fwd(y.view(b, T, DI), e["z"], wd["gnw"], DI)
    gb = binding.block_norm_bwd(n, e["res"], e["pre"], e["do"], e["dh"])
    dy, dz, _ = binding.gated_norm_bwd(y.view(b, T, DI), e["z"], wd["gnw"], gb["x"], DI)
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
    flat = lambda v: np.asarray(torch.as_tensor(v).double()).reshape(b * T, -1)  # noqa: E731
    rn, _ = gated_rmsnorm_fwd(flat(ry), flat(z), f["gnw"], 1e-5, DI)
    rb = layer.block_norm_bwd(rn, flat(res), pre, flat(do), flat(dh))
    rdy, rdz, _ = gated_rmsnorm_bwd(flat(ry), flat(z), f["gnw"], 1e-5, DI, rb["x"])
    t64 = lambda v: torch.as_tensor(np.asarray(v, dtype=np.float64))  # noqa: E731
    rs = ssd_grads(t64(ox), dt, w["dt_bias"], w["A"], t64(oB), t64(oC), w["D"],
                   t64(rdy).reshape(b, T, H, P))
    rc = layer.conv_bwd(xbc, w["cw"], np.concatenate([np.asarray(rs[k]).reshape(b, T, -1)
                                                      for k in ("x", "B", "C")], -1), w["cb"])
    for what, got, want in (("dresidual", gb["residual"], rb["residual"].reshape(b, T, DI)),
                            ("dz", dz, rdz.reshape(b, T, DI)), ("ddt", gs["dt"], rs["dt"]),
                            ("dxbc", gc["x"], rc["x"]), ("dweight", gc["weight"], rc["weight"]),
                            ("dbias", gc["bias"], rc["bias"])):
        err = rel_l2(got, want)
        print(f"  {what}: {err:.2e} of {TOL:.2e}", flush=True)
        assert err <= TOL, what
