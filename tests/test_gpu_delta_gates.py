"""Gradients of bf16 gates over many tokens (more than 65536 tokens times heads, whose backward
keeps the states rounded) where keys are alike and nothing or little decays."""
import numpy as np
import pytest
import torch

from oracle import delta
from state_space_model_ssd_amd import binding
from tests.delta_cases import dev, draw, unit
from tests.helpers import f64

pytestmark = pytest.mark.gpu

RMS = 2.0 ** -8 / 3 ** 0.5        # of one rounding to bf16: at most half a step, 2^-8, evenly spread
SCALE = 64 ** -0.5


def make(kind):
    """Keys alike (0.16 apart), close (0.02) or the same; no decay; beta 0.9 to 1, or 1; or neither."""
    x = draw(1, 2112, 32, 4, 32, 64, "bf16", "bf16", init=False, seed=12)
    assert x["g"].numel() > 65536
    r = torch.Generator().manual_seed(13)
    apart = {"alike": 0.02, "close": 0.0025, "same": 0.0}.get(kind.split()[0])
    if apart is not None:
        spread = apart * torch.randn(x["k"].shape, generator=r)
        x["k"] = unit(x["k"][:, :1].float() + spread).to(x["k"].dtype).expand_as(x["k"]).contiguous()
    if "keep" in kind:
        x["g"].zero_()
    x["beta"].copy_(1.0 if "one" in kind else 0.9 + 0.1 * x["beta"].float() if "high" in kind else
                    0.05 + 0.95 * x["beta"].float())
    dout = torch.randn(x["v"].shape, generator=r).to(x["v"].dtype)
    return x, dout


KINDS = ["spread", "keep one", "alike keep high", "alike keep one", "alike one", "close keep one",
         "close one", "same keep one"]


@pytest.mark.parametrize("kind", KINDS)
def test_beta(kind):
    """dbeta is the sum over the values of dR r, of which each is rounded to bf16 once, and rounded
    itself; the products' errors are independent, so their squares add up."""
    x, dout = make(kind)
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"])
    ref = delta.delta_bwd(*args, dout, SCALE)
    beta = f64(x["beta"])[..., None]
    terms = ref["v"] / beta * (delta.delta_fwd(*args, SCALE)[2] / beta)
    assert np.allclose(terms.sum(-1), ref["beta"])
    got = binding.delta_bwd(**dev(x), dout=dout.cuda())
    size = np.linalg.norm(ref["beta"])
    bound = RMS * (2 * np.linalg.norm(terms) ** 2 + size ** 2) ** 0.5
    err = np.linalg.norm(f64(got["beta"]) - ref["beta"])
    print(f"  dbeta: error {err:.3e}, bound {bound:.3e}, of {size:.3e}", flush=True)
    assert err <= bound


def decay_bound(x, dout):
    """What the roundings of kept values leave of dg, in the 2-norm.  dg of token i is <dS', A> with
    the decayed state A before it and its gradient dS'.  The state S entering i's 64 tokens is
    rounded, of which A has exp(G_i) S; the gradient dS of the state leaving them, which meets
    exp(G_64 - G_i) A; the rows r before i, of which A has beta exp(G_i - G_c) r k^T; and dg."""
    q, k, v, g, beta, do = (f64(t)[0] for t in (x["q"], x["k"], x["v"], x["g"], x["beta"], dout))
    T, H, P = v.shape
    rep = H // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    A, r, S = [], np.empty_like(v), np.zeros((H, P, q.shape[-1]))
    for t in range(T):
        A.append(S * np.exp(g[t])[:, None, None])
        r[t] = v[t] - (A[t] @ k[t][..., None])[..., 0]
        S = A[t] + (beta[t][:, None] * r[t])[..., None] * k[t][:, None]
    dg, squares = np.empty((T, H)), np.empty((T, H))
    G = np.empty_like(g)
    for s in range(0, T, 64):
        G[s:s + 64] = np.cumsum(g[s:s + 64], 0)
    dS = np.zeros_like(S)
    for t in reversed(range(T)):
        s, e = t - t % 64, min(t - t % 64 + 64, T)
        if t == e - 1:
            left = dS
        dS = dS + SCALE * do[t][..., None] * q[t][:, None]
        d = dS - (beta[t][:, None] * (dS @ k[t][..., None])[..., 0])[..., None] * k[t][:, None]
        dg[t] = (d * A[t]).sum((1, 2))
        S0 = A[s] * np.exp(-g[s])[:, None, None]
        one = np.exp(2 * G[t]) * ((d * S0) ** 2).sum((1, 2))
        two = np.exp(2 * (G[e - 1] - G[t])) * ((left * A[t]) ** 2).sum((1, 2))
        D = beta[s:t] * np.exp(G[t] - G[s:t])                                  # [c][h]
        rows = np.swapaxes(r[s:t], 0, 1) * (D.T[..., None] * (np.swapaxes(k[s:t], 0, 1) @ np.swapaxes(d, 1, 2)))
        squares[t] = one + two + (rows ** 2).sum((1, 2)) + dg[t] ** 2
        dS = d * np.exp(g[t])[:, None, None]
    return dg, RMS * squares.sum() ** 0.5


@pytest.mark.parametrize("kind", KINDS)
def test_decay(kind):
    """dg where it is of the size of its terms and where it is a small difference of them (keys
    alike and beta 1: what a token decays is overwritten)."""
    x, dout = make(kind)
    dg, bound = decay_bound(x, dout)
    got = binding.delta_bwd(**dev(x), dout=dout.cuda())
    size, err = np.linalg.norm(dg), np.linalg.norm(f64(got["g"])[0] - dg)
    print(f"  dg: error {err:.3e}, bound {bound:.3e}, of {size:.3e}", flush=True)
    assert err <= bound
